// Chunk plans: what octo_chunk_plan lays out and the chunk attention kernels read.
#pragma once

#include <vector>

#include "internal.h"

namespace octo {

// Keys of one segment's tokens [c W, c W + W), W the plan's block width, with the visibility that
// these 32 bytes give.  Slot j is token c W + j.  The row with own index i (at position p) sees it
// iff  lo <= j < hi  &&  own0 + j <= i  and
//     without a window  seen <= i,
//     under one         seen + j > p - window.
// own0 is kFarOwn where no order between row and key counts (an ancestor's or a mounted token).
// `seen` is the own index from which on rows see the block (a mount's point); under a window slot
// 0's position, or kSinkPos where the tokens are sinks: there a run of tokens whose positions jump,
// and one that the sinks end in, makes two blocks.
struct ChunkBlock {
  int32_t page[4];   // pages of slots [0, s), [s, 2 s) ..., s = min(page_size, W)
  int32_t own0, seen;
  uint16_t lo, hi;
  int32_t slot0;     // slot 0's place in its page (page 128: 0 or 64)
};

constexpr int32_t kFarOwn = -(1 << 30);
constexpr int32_t kSinkPos = 1 << 30;
constexpr int32_t kMaxPos = 1 << 29;   // positions of a chunk plan: their differences and the above fit 32 bits

// A piece of work: blocks [blk, blk + n) of kv head g for rows [row0, row0 + rows) of the plan.  Rows of
// one cursor: tokens from own index t0 on, under a window at positions own index + shift.  Or of
// several cursors next to each other, with blocks that all of them see (t0 = 0).  part < 0: all that
// the rows see, the result is written; else partial results from the part-th on (rows * G of them).
struct ChunkWork {
  int32_t row0, rows, t0, shift;
  int32_t blk, n, g, part;
};

// A joined piece of rows of kv head g: partial results refs[ref0 .. + n_refs), the first row's.
struct ChunkJoin {
  int32_t row0, rows, g, ref0, n_refs;
};

struct ChunkPlan {
  int32_t Hq = 0, G = 0, width = 0;   // width: keys per block
  int32_t tokens = 0;                 // tokens of 128 rows (of G heads each); a tile has up to twice as many
  int32_t window = 0;                 // 0: none
  bool tc = false;                    // tcgen05 kernels
  int32_t n_work = 0, n_joins = 0;
  int32_t n_ctas = 0;                 // tcgen05 kernels: CTAs, each with a run of the work
  int32_t max_rows = 0;               // rows of the longest tile
  int32_t max_join_rows = 0;          // and of the longest joined one
  int32_t max_refs = 0;
  int64_t n_part = 0;                 // partial results
  int64_t simt_ctas[9] = {};          // CUDA-core kernels: CTAs with work if each has 16 x rows
  ChunkBlock* blocks = nullptr;       // device arrays, the plan's
  ChunkWork* work = nullptr;          // CUDA-core kernels: longest first
  int32_t* cta_work = nullptr;        // [n_ctas + 1]
  ChunkJoin* joins = nullptr;
  int32_t* refs = nullptr;
  int32_t* drafted = nullptr;         // rows but the cursors' last ones
  int32_t* d_live = nullptr;          // [cursors + 1] cursors with rows before each
  std::vector<int32_t> row0, live;    // [cursors + 1] first row of each, d_live (host)
};

struct ChunkArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;        // may be NULL
  float scale;
  float* part;       // partial results: O [n_part][head_dim]
  float* part_ml;    // and (maximum, sum), in the log2 domain
};

bool chunk_tc_supported(const octo_pool_desc& d, int32_t width);
int chunk_tc(const octo_plan_s* p, const ChunkArgs& a, cudaStream_t s);
int chunk_simt(const octo_plan_s* p, const ChunkArgs& a, cudaStream_t s);
int chunk_join(const octo_plan_s* p, const ChunkArgs& a, cudaStream_t s);

}  // namespace octo
