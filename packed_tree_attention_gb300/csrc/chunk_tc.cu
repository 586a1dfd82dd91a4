// Chunk attention on the 5th-generation tensor cores (tcgen05, sm_103a): bf16 pools, blocks of
// 64 keys.
//
// Octopus project page, "Architecture & Co-Design" item 01 (Runtime): a turn's new tokens read
// the cursor's shared pages.  The query heads of a kv head read the same K and V, so a tile's
// 128 rows are T = 128 / G tokens times their G heads (row t G + h): a chunk of five tokens of
// four heads fills 20 of them and reads its context once, a prefill chunk fills all.  Plans with
// long chunks have tiles of twice as many: two slots of 128 rows that share each block of K and V.
// One CTA an SM, each with its share of the plan's work, pieces of tiles one after another; K and V
// come through a ring of blocks, S = Q K^T and O += P V are issued by threads of their own, a row
// of the softmax is a thread's.  Its running maximum stays until a block's probabilities relative
// to it sum past 2^16; the sum is kept in fp32 of the unrounded probabilities, P is rounded to
// bf16 (half a step, as the inputs' type has it).
//   k_chunk_stream  one slot.  Bound by HBM (32 KB a block and SM in 0.8 us), so nothing pauses at
//                   the end of a piece: the ring fills across it, S of the next one's first block
//                   is computed while the results are written.
//   k_chunk_pair    two slots.  Bound by the chain from S to S (0.82 us a block; the MMAs alone
//                   0.5 at 2.07 GHz), in which every wait and every instruction of the issuing
//                   threads counts: pieces start afresh, with the shortest loops.
// Partial results are joined by k_chunk_join.

#include <cuda_bf16.h>

#include "chunk.h"
#include "row_ring.cuh"
#include "tc_common.cuh"

namespace octo {
namespace {

using namespace tc;

template <int D, int kSlots>
struct Shape {
  static constexpr int kThreads = 128 + 128 * kSlots;
  static constexpr int kChunks = D / 64;                          // 128-byte columns of a row
  static constexpr uint32_t kQSlot = kChunks * 128 * 128;
  static constexpr uint32_t kTile = kChunks * 64 * 128;           // K or V of a block
  static constexpr uint32_t kStage = 2 * kTile;
  // what Q leaves of the SM's shared memory: some 190 KB under way for one slot, 160 for two
  static constexpr int kStages = kSlots == 2 ? (D == 128 ? 5 : 10) : (D == 128 ? 6 : 12);
  static constexpr uint32_t kOffKV = kSlots * kQSlot;
  static constexpr uint32_t kOffBar = kOffKV + kStages * kStage;
  static constexpr uint32_t kSmem = kOffBar + 512 + 1024;
  // TMEM columns: O, then S and P (one slot: 64, 2 x 32; two: 2 x 64 each, P over S)
  static constexpr uint32_t kColO = 0, kColS = kSlots * 128, kColP = 192;
  static constexpr uint32_t kCols = 256 * kSlots;
  static constexpr uint32_t kIdS = idesc_bf16(128, 64, 0, 0);
  static constexpr uint32_t kIdO = idesc_bf16(128, D, 0, 1);
};

struct TcParams {
  const ChunkBlock* blocks;
  const ChunkWork* work;
  const int32_t* cta_work;
  __nv_bfloat16* out;
  float *lse, *part, *part_ml;
  int32_t Hq, Hkv, G, P, T, box, loads, window;   // box: tokens of a query load; loads: of 64 keys
  float scale_log2;
  bool wide;                                      // out and part on 32-byte boundaries
  int32_t* status;
};

// Barriers of the two kernels, up to 512 bytes.
template <int kStages>
struct StreamBars {
  uint64_t q_full, q_free;   // queries loaded; no S of the piece to come
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t s_full, s_free;
  uint64_t p_full[2], o_done[2];
  uint64_t o_free;           // a piece's results have been read
  uint64_t drain;
  uint32_t tmem_base;
  volatile int32_t abort;
};
template <int kStages>
struct PairBars {
  uint64_t q_full;
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2];   // [slot][buffer]
  uint64_t drain;
  uint32_t tmem_base;
  volatile int32_t abort;
  __device__ void invalidate() {
    for (uint64_t* b = &q_full; b <= &drain; b++) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
  }
};

template <class B>
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, B* b, int32_t* status) {
  if (mbar_test(bar, parity)) return true;
  for (uint32_t i = 0; i < kSpinLimit; i++) {
    if (mbar_try(bar, parity)) return true;
    if ((i & 1023) == 1023 && b->abort) return false;
  }
  b->abort = 1;
  atomicExch(status, OCTO_ETIMEOUT);
  return false;
}
// For the copying threads, which are blocks ahead: their polls would take issue slots and shared
// memory cycles from the softmax (prefill 842 us with polls as above, 820 with these).
template <class B>
__device__ __forceinline__ bool wait_ahead(uint64_t* bar, uint32_t parity, B* b, int32_t* status) {
  for (uint32_t i = 0; i < (1u << 25); i++) {
    if (mbar_test(bar, parity)) return true;
    if ((i & 63) == 63 && b->abort) return false;
    __nanosleep(100);
  }
  b->abort = 1;
  atomicExch(status, OCTO_ETIMEOUT);
  return false;
}
// warp-uniform: the tcgen05 .sync.aligned accesses that follow need the whole warp
template <class B>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, B* b, int32_t* status) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, b, status));
}

// Stores n 32-bit words; wide: 32 bytes at a time, a whole sector of L2 (a warp's rows are far
// apart, and 16 bytes of each cost as many store cycles: 4 us for a tile's partial results).
template <int n>
__device__ __forceinline__ void store_words(void* dst, const uint32_t (&v)[n], bool wide) {
  uint32_t* d = static_cast<uint32_t*>(dst);
  if (wide) {
#pragma unroll
    for (int i = 0; i < n; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d + i), "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]),
                   "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < n; i += 4) st_global_v4(d + i, v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}

// A finished piece's row of this thread: O (TMEM column tO of its lane on) with its sum l and
// reference m, to the partial result `at` (>= 0) or, divided, to row `row` of the output.
template <int D>
__device__ __forceinline__ void write_row(const TcParams& p, uint32_t tO, bool live, int64_t at, size_t row, float m, float l) {
  const float inv = 1.f / l;
#pragma unroll 1
  for (int c = 0; c < D / 32; c++) {
    uint32_t o[32];
    tmem_ld32(tO + c * 32, o);
    tmem_wait_ld();
    if (live && at >= 0) {
      store_words(p.part + at * D + c * 32, o, p.wide);
    } else if (live) {
      uint32_t v[16];
#pragma unroll
      for (int i = 0; i < 16; i++) v[i] = pack_bf16(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
      store_words(p.out + row * D + c * 32, v, p.wide);
    }
  }
  if (live && at >= 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(m, l);
  else if (live && p.lse) p.lse[row] = (m + log2f(l)) * 0.69314718055994531f;
}

__device__ __forceinline__ ChunkWork load_work(const ChunkWork* w) {
  ChunkWork r;
  reinterpret_cast<int4*>(&r)[0] = reinterpret_cast<const int4*>(w)[0];
  reinterpret_cast<int4*>(&r)[1] = reinterpret_cast<const int4*>(w)[1];
  return r;
}

// The copies' run of work, one piece after another, its blocks' pages fetched 32 at a time, a lane each, and
// one such batch ahead (the next piece's first one at the last of this piece's): a load for each
// block as it comes would make every block wait for memory, some 1 to 3 us in a streaming kernel.
// All lanes call it alike.
struct Feed {
  struct Pages {
    int4 page;
    int slot0;
  };
  const ChunkWork* work;
  const ChunkBlock* blocks;
  int i, end;           // the piece at hand, the run's end
  ChunkWork w, w1;      // this piece and the next
  Pages cur, ahead;
  __device__ __forceinline__ Pages fetch(const ChunkWork& x, int j) const {
    const ChunkBlock* b = blocks + x.blk + min(j + (int)(threadIdx.x & 31), x.n - 1);
    return {*reinterpret_cast<const int4*>(b->page), b->slot0};
  }
  __device__ __forceinline__ void start(const ChunkWork* wk, const ChunkBlock* b, int w0, int we) {
    work = wk, blocks = b, i = w0, end = we;
    w = load_work(work + i);
    w1 = load_work(work + min(i + 1, end - 1));
    ahead = fetch(w, 0);
  }
  // before block j of the piece: its pages are in lane j % 32's `cur`
  __device__ __forceinline__ void at(int j) {
    if (j % 32 == 0) {
      cur = ahead;
      ahead = j + 32 < w.n ? fetch(w, j + 32) : fetch(w1, 0);
    }
  }
  // to the next piece (before any at() of it)
  __device__ __forceinline__ void step() {
    i++;
    w = w1;
    w1 = load_work(work + min(i + 1, end - 1));
  }
};

// Warps: 0 copies K and V, 2 allocates TMEM and copies Q, 1 issues the MMAs, 4-7 are the softmax.
// S has one buffer, free again as soon as the softmax has it in registers, and P two of its own:
// S of the next block waits neither for the softmax nor behind P V (P over S in two buffers, S two
// blocks ahead but behind P V: 64 cursors' drafts 137 us where these take 128).  Warps whose rows
// a tile does not have only keep step.
template <int D>
__global__ void __launch_bounds__(Shape<D, 1>::kThreads, 1)
    k_chunk_stream(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TcParams p) {
  using S = Shape<D, 1>;
  constexpr int kNS = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto* B = reinterpret_cast<StreamBars<kNS>*>(smem + S::kOffBar);
  static_assert(sizeof(StreamBars<kNS>) <= 512, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  rows::launch_dependents();   // they wait for this grid's end before they touch its results
  const int w0 = p.cta_work[blockIdx.x], w1 = p.cta_work[blockIdx.x + 1];   // at least one piece, of at least one block

  if (threadIdx.x == 0) {
    mbar_init(&B->q_full, 1);
    mbar_init(&B->q_free, 1);
    for (int s = 0; s < kNS; s++) {
      mbar_init(&B->kv_full[s], 1);
      mbar_init(&B->kv_empty[s], 1);
    }
    mbar_init(&B->s_full, 1);
    mbar_init(&B->s_free, 4);          // the softmax warps
    for (int b = 0; b < 2; b++) {
      mbar_init(&B->p_full[b], 4);
      mbar_init(&B->o_done[b], 1);
    }
    mbar_init(&B->o_free, 4);
    mbar_init(&B->drain, 1);
    B->abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&B->tmem_base, S::kCols);
    tmem_relinquish();
  }
  // rows of the tiles that no query load writes: finite, for the warps that have rows besides
  {
    const int q_rows = p.box * p.G;
    for (int c = 0; c < S::kChunks; c++)
      for (int i = q_rows * 8 + threadIdx.x; i < 128 * 8; i += S::kThreads)
        *reinterpret_cast<uint4*>(smem + c * 16384 + i * 16) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = B->tmem_base;
  const uint32_t sQ = smem_u32(smem), sKV = smem_u32(smem + S::kOffKV);

  if (warp == 0) {
    // ---------------- copies of K and V ----------------
    if (lane == 0) {
      prefetch_map(&tmK);
      prefetch_map(&tmV);
    }
    Feed f;
    f.start(p.work, p.blocks, w0, w1);
    rows::wait_for_predecessor();
    const uint32_t part = 8192u / p.loads;   // bytes of a load
    int st = 0, issued = 0;
    uint32_t round = 0;                      // parity of the ring's rounds
    bool ok = true;
    for (; ok && f.i < w1; f.step()) {
      for (int j = 0; j < f.w.n; j++) {
        f.at(j);
        int page[4];
        page[0] = __shfl_sync(0xffffffffu, f.cur.page.x, j % 32);
        page[1] = __shfl_sync(0xffffffffu, f.cur.page.y, j % 32);
        page[2] = __shfl_sync(0xffffffffu, f.cur.page.z, j % 32);
        page[3] = __shfl_sync(0xffffffffu, f.cur.page.w, j % 32);
        const int slot0 = __shfl_sync(0xffffffffu, f.cur.slot0, j % 32);
        if (issued >= kNS && !(ok = warp_wait(&B->kv_empty[st], round ^ 1, B, p.status))) break;
        if (lane == 0) {
          uint8_t* dst = smem + S::kOffKV + st * S::kStage;
          mbar_expect_tx(&B->kv_full[st], S::kStage);
#pragma unroll
          for (int l = 0; l < 4; l++) {
            if (l >= p.loads) break;
            const int row = (page[l] * p.Hkv + f.w.g) * p.P + slot0;
#pragma unroll
            for (int c = 0; c < S::kChunks; c++) {
              tma_load_2d(dst + c * 8192 + l * part, &tmK, &B->kv_full[st], c * 64, row);
              tma_load_2d(dst + S::kTile + c * 8192 + l * part, &tmV, &B->kv_full[st], c * 64, row);
            }
          }
        }
        __syncwarp();
        issued++;
        if (++st == kNS) st = 0, round ^= 1;
      }
    }
    // every copy that was started has landed before the CTA may exit
    if (lane == 0)
      for (int j = max(0, issued - kNS); j < issued; j++)
        mbar_wait(&B->kv_full[j % kNS], (j / kNS) & 1, p.status, OCTO_ETIMEOUT);
    __syncwarp();
  } else if (warp == 2) {
    // ---------------- copies of Q ----------------
    if (lane == 0) {
      prefetch_map(&tmQ);
      ChunkWork w = load_work(p.work + w0), next = w;
      rows::wait_for_predecessor();
      int i = w0;
      for (; i < w1; i++, w = next) {
        if (i + 1 < w1) next = load_work(p.work + i + 1);
        if (i > w0 && !wait_ahead(&B->q_free, (i - w0 - 1) & 1, B, p.status)) break;
        mbar_expect_tx(&B->q_full, (uint32_t)(S::kChunks * p.box * p.G * 128));
        for (int c = 0; c < S::kChunks; c++) tma_load_3d(smem + c * 16384, &tmQ, &B->q_full, c * 64, w.g * p.G, w.row0);
      }
      mbar_wait(&B->q_full, (i - w0 - 1) & 1, p.status, OCTO_ETIMEOUT);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMAs ----------------
    if (lane == 0) {
      const uint64_t dq0 = desc_sw128(sQ, 16, 1024);
      const uint64_t dk0 = desc_sw128(sKV, 16, 1024);
      const uint64_t dv0 = desc_sw128(sKV + S::kTile, 8192, 1024);
      const uint32_t dO = tbase + S::kColO, dS = tbase + S::kColS, dP = tbase + S::kColP;
      auto issue_S = [&](int st) {
        const uint64_t kb = dk0 + (uint64_t)(st * (S::kStage >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; kk++) {
          const uint32_t qo = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          const uint32_t ko = ((kk >> 2) * 8192 + (kk & 3) * 32) >> 4;
          mma_f16_ss(dS, dq0 + qo, kb + ko, S::kIdS, kk > 0);
        }
        mma_commit(&B->s_full);
      };
      auto issue_PV = [&](int st, int b, bool first) {
        const uint64_t vb = dv0 + (uint64_t)(st * (S::kStage >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; kk++)
          mma_f16_ts(dO, dP + b * 32 + kk * 8, vb + (uint64_t)(kk * (2048 >> 4)), S::kIdO, (!first || kk > 0) ? 1u : 0u);
        mma_commit(&B->o_done[b]);
        mma_commit(&B->kv_empty[st]);
      };
      int st = 0;                // ring stage of the block at hand
      uint32_t round = 0;
      auto next_stage = [&] {
        if (++st == kNS) st = 0, round ^= 1;
      };
      int cnt = 0, pieces = 0;   // this slot's blocks and pieces
      bool ok = true;
      ChunkWork w = load_work(p.work + w0), next = w;
      for (int i = w0; ok && i < w1; i++, w = next) {
        if (i + 1 < w1) next = load_work(p.work + i + 1);
        if (!(ok = wait_or_abort(&B->q_full, (i - w0) & 1, B, p.status))) break;
        // the S buffer is free: P of the block before was waited for
        if (!(ok = wait_or_abort(&B->kv_full[st], round, B, p.status))) break;
        tc_fence_after();
        issue_S(st);
        for (int j = 0; j < w.n; j++, cnt++) {
          const int at = st;
          next_stage();
          if (j + 1 < w.n) {
            if (!(ok = wait_or_abort(&B->kv_full[st], round, B, p.status))) break;
            if (!(ok = wait_or_abort(&B->s_free, cnt & 1, B, p.status))) break;
            tc_fence_after();
            issue_S(st);
          } else {
            mma_commit(&B->q_free);
          }
          if (!(ok = wait_or_abort(&B->p_full[cnt & 1], (cnt >> 1) & 1, B, p.status))) break;
          // the results in O have been read before this piece's replace them
          if (j == 0 && pieces > 0 && !(ok = wait_or_abort(&B->o_free, (pieces - 1) & 1, B, p.status))) break;
          tc_fence_after();
          issue_PV(at, cnt & 1, j == 0);
        }
        pieces++;
      }
      // all MMAs of this thread are complete before TMEM is released
      mma_commit(&B->drain);
      mbar_wait(&B->drain, 0, p.status, OCTO_ETIMEOUT);
    }
  } else if (warp >= 4) {
    // ---------------- softmax ----------------
    const int wq = warp & 3;
    const int r = wq * 32 + lane;
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tbase + lane_off + S::kColS, tP = tbase + lane_off + S::kColP;
    const uint32_t tO = tbase + lane_off + S::kColO;
    const bool windowed = p.window > 0;
    const int tok_r = r / p.G, h_r = r - tok_r * p.G;
    ChunkWork w = load_work(p.work + w0), next = w;
    // own0, seen, lo | hi << 16 of this block, the next and the one after
    auto fields = [&](const ChunkWork& x, int j) { return *reinterpret_cast<const int4*>(&p.blocks[x.blk + min(j, x.n - 1)].own0); };
    int4 e, e1, e2;
    int before = 0;   // blocks of the piece before
    int cnt = 0;
    bool ok = true;
    for (int i = w0; ok && i < w1; i++, w = next) {
      if (i + 1 < w1) next = load_work(p.work + i + 1);
      if (before < 2) e1 = fields(w, 0), e2 = fields(w, 1);
      const int R = w.rows * p.G;
      before = w.n;
      const bool mine = wq * 32 < R;
      // own index of this thread's row, and of the warp's first and last one
      const int own = w.t0 + tok_r;
      const int own_first = w.t0 + wq * 32 / p.G, own_last = w.t0 + min(wq * 32 + 31, R - 1) / p.G;
      const int w_shift = w.shift - p.window + 1;
      float m_used = -INFINITY, l = 0.f;
      for (int j = 0; j < w.n; j++, cnt++) {
        e = e1, e1 = e2;
        e2 = j + 2 < w.n ? fields(w, j + 2) : fields(next, j + 2 - w.n);
        const int b = cnt & 1;
        if (!(ok = warp_wait(&B->s_full, cnt & 1, B, p.status))) break;
        if (mine) {
          int lo = e.z & 0xffff, hi = (uint32_t)e.z >> 16;
          const bool full = lo == 0 && hi == 64 && e.x + 63 <= own_first && (windowed ? own_last + w_shift <= e.y : e.y <= own_first);
          tc_fence_after();
          uint32_t s0[32], s1[32];
          tmem_ld32(tS, s0);
          tmem_ld32(tS + 32, s1);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&B->s_free);
          float x[64];   // raw scores; the scale is folded into the exponent
#pragma unroll
          for (int k = 0; k < 32; k++) {
            x[k] = __uint_as_float(s0[k]);
            x[32 + k] = __uint_as_float(s1[k]);
          }
          if (!full) {
            if (windowed) lo = max(lo, own + w_shift - e.y);
            else if (own < e.y) lo = 64;
            hi = min(hi, own - e.x + 1);
#pragma unroll
            for (int k = 0; k < 64; k++)
              if (k < lo || k >= hi) x[k] = -INFINITY;
          }
          bool need = false;
          float factor = 1.f;
          // nothing visible to this row yet: start from the block's exact maximum
          if (m_used == -INFINITY) m_used = max64(x) * p.scale_log2;
          float msub = (m_used == -INFINITY) ? 0.f : m_used;
          uint32_t pk[32];
          auto pass = [&]() -> float {
            float ps[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 32; k++) {
              float a, c;
              fma2(a, c, x[2 * k], x[2 * k + 1], p.scale_log2, -msub);
              a = ex2(a);
              c = ex2(c);
              add2(ps[2 * (k & 3)], ps[2 * (k & 3) + 1], ps[2 * (k & 3)], ps[2 * (k & 3) + 1], a, c);
              pk[k] = pack_bf16(a, c);
            }
            return ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
          };
          float le = pass();
          const bool over = !(le <= 65536.f);
          if (__any_sync(0xffffffffu, over)) {
            if (over) {
              const float mc = max64(x) * p.scale_log2;
              factor = ex2(m_used - mc);
              l *= factor;
              m_used = mc;
              msub = mc;
              need = true;
            }
            le = pass();
          }
          l += le;
          if (j > 0 && __any_sync(0xffffffffu, need)) {
            // O must hold every P V so far before it is rescaled
            if (!(ok = warp_wait(&B->o_done[(cnt - 1) & 1], ((cnt - 1) >> 1) & 1, B, p.status))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; c++) {
              uint32_t ov[32];
              tmem_ld32(tO + c * 32, ov);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; k++) ov[k] = __float_as_uint(__uint_as_float(ov[k]) * factor);
              tmem_st32(tO + c * 32, ov);
            }
            tmem_wait_st();
          }
          // P V of the block before the last has read this buffer: S, issued after it, is here
          tmem_st32(tP + b * 32, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
        } else if (lane == 0) {
          mbar_arrive(&B->s_free);
        }
        if (lane == 0) mbar_arrive(&B->p_full[b]);
      }
      // ---------------- results ----------------
      if (!ok || !(ok = warp_wait(&B->o_done[(cnt - 1) & 1], ((cnt - 1) >> 1) & 1, B, p.status))) break;
      if (mine) {
        tc_fence_after();
        write_row<D>(p, tO, r < R, w.part >= 0 ? (int64_t)w.part + r : -1, (size_t)(w.row0 + tok_r) * p.Hq + w.g * p.G + h_r, m_used, l);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->o_free);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tbase, S::kCols);
}

// Warps: 0 copies Q, K and V, 2 allocates TMEM, 1 and 3 issue the MMAs of slots 0 and 1, 4-7 and
// 8-11 are the slots' softmax.  S has two buffers a slot and is issued two blocks ahead; P goes
// over the S that it came from, and S of the block after the next into that buffer behind P V, in
// the order of the issuing thread.  Tried and slower at prefill: S a block ahead with P beside it
// (872 us for 826), a thread for P V (1,110), the slots' exponentials in strict turns (979), every
// fourth exponential by a polynomial on the FMA pipe (858 for 841), the scores in two halves (857).
template <int D>
__global__ void __launch_bounds__(Shape<D, 2>::kThreads, 1)
    k_chunk_pair(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TcParams p) {
  using S = Shape<D, 2>;
  constexpr int kSlots = 2;
  constexpr int kNS = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  auto* B = reinterpret_cast<PairBars<kNS>*>(smem + S::kOffBar);
  static_assert(sizeof(PairBars<kNS>) <= 512, "barriers");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  rows::launch_dependents();   // they wait for this grid's end before they touch its results
  const int w0 = p.cta_work[blockIdx.x], w1 = p.cta_work[blockIdx.x + 1];   // at least one piece, of at least one block
  if (warp == 2) {
    tmem_alloc(&B->tmem_base, S::kCols);
    tmem_relinquish();
  }
  // rows of the tile that no query load writes: finite, for the warps that have rows besides
  {
    const int q_rows = p.box * p.G;
    for (int s = 0; s < kSlots; s++)
      for (int c = 0; c < S::kChunks; c++)
        for (int x = q_rows * 8 + threadIdx.x; x < 128 * 8; x += S::kThreads)
          *reinterpret_cast<uint4*>(smem + s * S::kQSlot + c * 16384 + x * 16) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  const uint32_t sQ = smem_u32(smem), sKV = smem_u32(smem + S::kOffKV);

  ChunkWork next_work = load_work(p.work + w0);
#pragma unroll 1
  for (int i = w0; i < w1; i++) {
    const ChunkWork t = next_work;
    next_work = load_work(p.work + min(i + 1, w1 - 1));
    const int g = t.g, n = t.n;
    const ChunkBlock* blk = p.blocks + t.blk;
    const int n_slots = t.rows > p.T ? 2 : 1;
    auto slot_rows = [&](int s) { return min(t.rows - s * p.T, p.T) * p.G; };
    if (threadIdx.x == 0) {
      if (i > w0) B->invalidate();   // every phase of the piece before is over
      mbar_init(&B->q_full, 1);
      for (int s = 0; s < kNS; s++) {
        mbar_init(&B->kv_full[s], 1);
        mbar_init(&B->kv_empty[s], n_slots);   // released by the slots' P V
      }
      for (int h = 0; h < kSlots; h++)       // those of a slot without rows too: invalidate() takes all
        for (int b = 0; b < 2; b++) {
          mbar_init(&B->s_full[h][b], 1);
          mbar_init(&B->p_full[h][b], h < n_slots ? (slot_rows(h) + 31) / 32 * 32 : 1);
          mbar_init(&B->o_done[h][b], 1);
        }
      mbar_init(&B->drain, n_slots);
      if (i == w0) B->abort = 0;
      fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (B->abort) break;
    const uint32_t tbase = B->tmem_base;

    if (warp == 0) {
      // ---------------- copies ----------------
      if (lane == 0) {
        prefetch_map(&tmQ);
        prefetch_map(&tmK);
        prefetch_map(&tmV);
        if (i == w0) rows::wait_for_predecessor();
        mbar_expect_tx(&B->q_full, (uint32_t)(n_slots * S::kChunks * p.box * p.G * 128));
        for (int s = 0; s < n_slots; s++)
          for (int c = 0; c < S::kChunks; c++)
            tma_load_3d(smem + s * S::kQSlot + c * 16384, &tmQ, &B->q_full, c * 64, g * p.G, t.row0 + s * p.T);
        int issued = 0;
        const uint32_t part = 8192u / p.loads;   // bytes of a load
        ChunkBlock next = blk[0];
        for (int j = 0; j < n; j++) {
          const int st = j % kNS;
          const ChunkBlock k = next;
          if (j + 1 < n) next = blk[j + 1];      // off the critical path
          if (j >= kNS && !wait_ahead(&B->kv_empty[st], ((j / kNS) - 1) & 1, B, p.status)) break;
          uint8_t* dst = smem + S::kOffKV + st * S::kStage;
          mbar_expect_tx(&B->kv_full[st], S::kStage);
#pragma unroll
          for (int l = 0; l < 4; l++) {
            if (l >= p.loads) break;
            const int row = (k.page[l] * p.Hkv + g) * p.P + k.slot0;
#pragma unroll
            for (int c = 0; c < S::kChunks; c++) {
              tma_load_2d(dst + c * 8192 + l * part, &tmK, &B->kv_full[st], c * 64, row);
              tma_load_2d(dst + S::kTile + c * 8192 + l * part, &tmV, &B->kv_full[st], c * 64, row);
            }
          }
          issued = j + 1;
        }
        // every copy that this thread started has landed, and every slot of the ring has been given
        // back, before the barriers are made anew or the CTA ends
        mbar_wait(&B->q_full, 0, p.status, OCTO_ETIMEOUT);
        for (int j = max(0, issued - kNS); j < issued; j++) {
          mbar_wait(&B->kv_full[j % kNS], (j / kNS) & 1, p.status, OCTO_ETIMEOUT);
          wait_or_abort(&B->kv_empty[j % kNS], (j / kNS) & 1, B, p.status);
        }
      }
    } else if (warp == 1 || (warp == 3 && n_slots == 2)) {
      // ---------------- MMAs ----------------
      const int hh = warp == 1 ? 0 : 1;
      if (lane == 0) {
        const uint64_t dq0 = desc_sw128(sQ + hh * S::kQSlot, 16, 1024);
        const uint64_t dk0 = desc_sw128(sKV, 16, 1024);
        const uint64_t dv0 = desc_sw128(sKV + S::kTile, 8192, 1024);
        const uint32_t dO = tbase + S::kColO + hh * 128, dS = tbase + S::kColS + hh * 128;
        auto issue_S = [&](int st, int b) {
          const uint64_t kb = dk0 + (uint64_t)(st * (S::kStage >> 4));
#pragma unroll
          for (int kk = 0; kk < D / 16; kk++) {
            const uint32_t qo = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
            const uint32_t ko = ((kk >> 2) * 8192 + (kk & 3) * 32) >> 4;
            mma_f16_ss(dS + b * 64, dq0 + qo, kb + ko, S::kIdS, kk > 0);
          }
          mma_commit(&B->s_full[hh][b]);
        };
        auto issue_PV = [&](int st, int b, bool first) {
          const uint64_t vb = dv0 + (uint64_t)(st * (S::kStage >> 4));
#pragma unroll
          for (int kk = 0; kk < 4; kk++)
            mma_f16_ts(dO, dS + b * 64 + kk * 8, vb + (uint64_t)(kk * (2048 >> 4)), S::kIdO, (!first || kk > 0) ? 1u : 0u);
          mma_commit(&B->o_done[hh][b]);
        };
        bool ok = wait_or_abort(&B->q_full, 0, B, p.status);
        for (int j = 0; ok && j < min(n, 2); j++) {
          if (!(ok = wait_or_abort(&B->kv_full[j], 0, B, p.status))) break;
          tc_fence_after();
          issue_S(j, j);
        }
        for (int j = 0; ok && j < n; j++) {
          const int st = j % kNS, b = j & 1, j2 = j + 2;
          if (!(ok = wait_or_abort(&B->p_full[hh][b], (j >> 1) & 1, B, p.status))) break;
          tc_fence_after();
          issue_PV(st, b, j == 0);
          mma_commit(&B->kv_empty[st]);
          if (j2 < n) {
            // buffer b held P of block j, which P V above reads first (MMAs of a thread run in order)
            if (!(ok = wait_or_abort(&B->kv_full[j2 % kNS], (j2 / kNS) & 1, B, p.status))) break;
            tc_fence_after();
            issue_S(j2 % kNS, b);
          }
        }
        // all MMAs of this thread are complete before TMEM is released
        mma_commit(&B->drain);
        mbar_wait(&B->drain, 0, p.status, OCTO_ETIMEOUT);
      }
    } else if (warp >= 4 && ((warp - 4) >> 2) < n_slots && (warp & 3) * 32 < slot_rows((warp - 4) >> 2)) {
      // ---------------- softmax ----------------
      const int hh = (warp - 4) >> 2, wq = warp & 3;
      const int r = wq * 32 + lane, R = slot_rows(hh);
      const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
      const uint32_t tS0 = tbase + lane_off + S::kColS + hh * 128;
      const uint32_t tO = tbase + lane_off + S::kColO + hh * 128;
      // own index of this thread's row, and of the warp's first and last one
      const int base = t.t0 + hh * p.T;
      const int own = base + min(r, R - 1) / p.G;
      const int own_first = base + wq * 32 / p.G, own_last = base + min(wq * 32 + 31, R - 1) / p.G;
      const bool windowed = p.window > 0;
      const int w_shift = t.shift - p.window + 1;
      float m_used = -INFINITY, l = 0.f;
      bool ok = true;
      auto fields = [&](int j) { return *reinterpret_cast<const int4*>(&blk[j].own0); };   // own0, seen, lo | hi << 16, slot0
      int4 next = fields(0);
      for (int j = 0; j < n; j++) {
        const int4 e = next;
        if (j + 1 < n) next = fields(j + 1);
        const int b = j & 1;
        int lo = e.z & 0xffff, hi = (uint32_t)e.z >> 16;
        const bool full = lo == 0 && hi == 64 && e.x + 63 <= own_first && (windowed ? own_last + w_shift <= e.y : e.y <= own_first);
        if (!(ok = warp_wait(&B->s_full[hh][b], (j >> 1) & 1, B, p.status))) break;
        tc_fence_after();
        uint32_t s0[32], s1[32];
        tmem_ld32(tS0 + b * 64, s0);
        tmem_ld32(tS0 + b * 64 + 32, s1);
        tmem_wait_ld();
        float x[64];   // raw scores; the scale is folded into the exponent
#pragma unroll
        for (int i = 0; i < 32; i++) {
          x[i] = __uint_as_float(s0[i]);
          x[32 + i] = __uint_as_float(s1[i]);
        }
        if (!full) {
          if (windowed) lo = max(lo, own + w_shift - e.y);
          else if (own < e.y) lo = 64;
          hi = min(hi, own - e.x + 1);
#pragma unroll
          for (int i = 0; i < 64; i++)
            if (i < lo || i >= hi) x[i] = -INFINITY;
        }
        bool need = false;
        float factor = 1.f;
        // nothing visible to this row yet: start from the block's exact maximum
        if (m_used == -INFINITY) m_used = max64(x) * p.scale_log2;
        float msub = (m_used == -INFINITY) ? 0.f : m_used;
        uint32_t pk[32];
        auto pass = [&]() -> float {
          float ps[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 32; i++) {
            float a, c;
            fma2(a, c, x[2 * i], x[2 * i + 1], p.scale_log2, -msub);
            a = ex2(a);
            c = ex2(c);
            add2(ps[2 * (i & 3)], ps[2 * (i & 3) + 1], ps[2 * (i & 3)], ps[2 * (i & 3) + 1], a, c);
            pk[i] = pack_bf16(a, c);
          }
          return ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
        };
        float le = pass();
        const bool over = !(le <= 65536.f);
        if (__any_sync(0xffffffffu, over)) {
          if (over) {
            const float mc = max64(x) * p.scale_log2;
            factor = ex2(m_used - mc);
            l *= factor;
            m_used = mc;
            msub = mc;
            need = true;
          }
          le = pass();
        }
        l += le;
        if (j > 0 && __any_sync(0xffffffffu, need)) {
          // O must hold every P V so far before it is rescaled
          if (!(ok = warp_wait(&B->o_done[hh][(j - 1) & 1], ((j - 1) >> 1) & 1, B, p.status))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; c++) {
            uint32_t ov[32];
            tmem_ld32(tO + c * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i++) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * factor);
            tmem_st32(tO + c * 32, ov);
          }
          tmem_wait_st();
        }
        tmem_st32(tS0 + b * 64, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&B->p_full[hh][b]);
      }
      // ---------------- results ----------------
      // both buffers' last commits: an arrival still to come may not meet the barriers made anew
      if (ok && n > 1) ok = warp_wait(&B->o_done[hh][(n - 2) & 1], ((n - 2) >> 1) & 1, B, p.status);
      if (ok && warp_wait(&B->o_done[hh][(n - 1) & 1], ((n - 1) >> 1) & 1, B, p.status)) {
        tc_fence_after();
        const int tok = hh * p.T + min(r, R - 1) / p.G, h = min(r, R - 1) % p.G;
        write_row<D>(p, tO, r < R, t.part >= 0 ? (int64_t)t.part + tok * p.G + h : -1, (size_t)(t.row0 + tok) * p.Hq + g * p.G + h,
                     m_used, l);
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  if (warp == 2) tmem_dealloc(B->tmem_base, S::kCols);
}

template <int D, int kSlots>
int launch(const octo_plan_s* plan, const ChunkArgs& a, cudaStream_t s) {
  using S = Shape<D, kSlots>;
  const octo_pool_desc& d = plan->pool->desc;
  const ChunkPlan& c = *plan->chunk;
  TcParams p;
  p.blocks = c.blocks, p.work = c.work, p.cta_work = c.cta_work;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse, p.part = a.part, p.part_ml = a.part_ml;
  p.Hq = c.Hq, p.Hkv = d.n_kv_heads, p.G = c.G, p.P = d.page_size, p.T = c.tokens;
  p.box = c.max_rows < c.tokens ? c.max_rows : c.tokens;
  const int span = d.page_size < 64 ? d.page_size : 64;
  p.loads = 64 / span;
  p.window = c.window;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.wide = !(((uintptr_t)a.out | (uintptr_t)a.part) & 31);
  p.status = plan->pool->d_status;
  CUtensorMap mq, mk, mv;
  {
    uint64_t dims[3] = {(uint64_t)D, (uint64_t)c.Hq, (uint64_t)plan->info.n_rows};
    uint64_t str[2] = {D * 2, (uint64_t)c.Hq * D * 2};
    uint32_t box[3] = {64, (uint32_t)c.G, (uint32_t)p.box};
    if (int st = encode_tmap(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, str, box,
                             CU_TENSOR_MAP_SWIZZLE_128B))
      return st;
  }
  {
    uint64_t dims[2] = {(uint64_t)D, (uint64_t)d.num_pages * d.n_kv_heads * d.page_size};
    uint64_t str[1] = {D * 2};
    uint32_t box[2] = {64, (uint32_t)span};
    if (int st = encode_tmap(&mk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(a.k), dims, str, box,
                             CU_TENSOR_MAP_SWIZZLE_128B))
      return st;
    if (int st = encode_tmap(&mv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(a.v), dims, str, box,
                             CU_TENSOR_MAP_SWIZZLE_128B))
      return st;
  }
  const void* kernel = kSlots == 2 ? (const void*)k_chunk_pair<D> : (const void*)k_chunk_stream<D>;
  if (int st = set_smem_limit(kernel, (int)S::kSmem)) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)c.n_ctas);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  void* args[4] = {&mq, &mk, &mv, &p};
  OCTO_CUDA(cudaLaunchKernelExC(&cfg, kernel, args));
  count_launch();
  return OCTO_OK;
}

}  // namespace

bool chunk_tc_supported(const octo_pool_desc& d, int32_t width) {
  // rows of the pool arrays are a coordinate of the copies, 32 bits with a sign
  return d.dtype == OCTO_DTYPE_BF16 && width == 64 && (int64_t)d.num_pages * d.n_kv_heads * d.page_size <= INT32_MAX;
}

int chunk_tc(const octo_plan_s* plan, const ChunkArgs& a, cudaStream_t s) {
  const bool two = plan->chunk->max_rows > plan->chunk->tokens;
  if (plan->pool->desc.head_dim == 64) return two ? launch<64, 2>(plan, a, s) : launch<64, 1>(plan, a, s);
  return two ? launch<128, 2>(plan, a, s) : launch<128, 1>(plan, a, s);
}

}  // namespace octo
