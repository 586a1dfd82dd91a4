// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// With p_r = softmax(c x_r) the target's distribution after row r and q_r the draft's, the draft
// in row r + 1, token y, is accepted with probability a = min(1, p_r(y) / q_r(y)); after the
// first rejected one the next token is drawn from max(0, p_r - q_r) / sum, else from p.  A draw
// from weights w is argmax_v w_v / e_v with e_v ~ Exp(1) independent (the first of exponential
// clocks of rates w_v), so that neither a sum of the weights nor an order of them is needed.
//
//   k_verify_stats   softmax statistics of all rows, in equal runs over all SMs
//   k_verify_queue   the same where there are many cursors, but for most of what comes behind a
//                    cursor's first rejected draft
//   k_verify_decide  greedy: a CTA a cursor, the first rejected draft and the next token
//   k_verify_draw    sampled: the first rejected draft, then the race over one row (pair) of each
//                    cursor
// 256 cursors of five rows of 151,936 bf16 logits and four drafts' distributions (700 MB), 1.3
// drafts accepted on average: 136 us, of which the draw some 50; with k_verify_stats (106 us, 6.5
// TB/s) 161.  One cursor: 12.0, most of it the host's (the decision as a kernel of its own: 14.5).
// The sums are fp32 of fp32 exponentials; a decision turns where they are off by some 1e-7 of a
// probability, for the exponents that its ratio is made of are kept in two parts.

#include <algorithm>
#include <cmath>

#include "chunk.h"
#include "row_common.cuh"
#include "row_ring.cuh"

namespace octo {
namespace {

using namespace rows;

constexpr int kThreads = 512;
constexpr int kHeld = 2;              // CTAs of 512 threads that an SM holds
constexpr int kChunk = kPer * kThreads;   // vectors that a CTA takes at once, at most
constexpr int kDecide = 256;          // threads of a cursor's decision
constexpr int kSummers = kThreads - 32;   // of a CTA of k_verify_queue; its last warp is in control
constexpr int kAhead = 2;             // units that such a CTA holds
constexpr int kNone = 0x7fffffff;
// Probabilities below e^-745 are 0, as they are in 64 bits: a draft that the target masks by its type's
// lowest value is not taken because the draft's distribution masks it so too.
constexpr float kLogZero = -745.f;

// What is decided about a cursor: accepted drafts, the row (of the logits given) of the next
// token's distribution with its statistics, and what a rejected draft takes off it: the draft's
// distribution of that row (y_row >= 0) or one id (out >= 0).
struct Decision {
  int32_t acc, row, y_row, out;
  float2 st, y_st;
};

struct VerifyParams {
  const void *x, *y;          // target's and draft's logits
  int64_t ld, yld, eld;
  int32_t V;
  float c, cy;                // inverse temperatures
  float hi[2], lo[2];         // c log2 e and cy log2 e in two parts, lo > 0
  const int32_t* row0;        // [cursors + 1] first row of the plan's cursors, from cur0 on
  const int32_t* live;        // [cursors + 1] cursors with rows before each, from cur0 on
  const int32_t* drafted;     // rows of the plan that lead to a draft, from the first of these on
  int32_t first, live0;       // row0[0], live[0]
  const int32_t* ids;
  const float *u, *noise;
  int32_t *n_accept, *next_id;
  float *next_logp, *accept_p;
  float2* stat;               // [n_rows + n_drafted][slots] (m, S) of the target's and the draft's rows
  unsigned long long* best;   // [n_rows][slots] greedy: order_key of the largest logit, ~id
  unsigned long long* drawn;  // [n_cur] best score
  int32_t* done;              // [n_cur] CTAs that are through with the cursor's draw
  int32_t* rejected;          // [n_cur] first rejected draft so far, kNone: none
  int32_t* parts_done;        // [n_rows] units of the row, and of the draft's, that are summed
  int32_t* ticket;            // the next unit but the first ones of all CTAs
  int32_t n_rows, n_drafted, n_cur;
  int32_t per_row, per_chunk, slots, ctas;   // chunks of a row, vectors of a chunk
  int32_t longest;            // rows of the longest cursor
  int32_t parts, units;       // queue: units of a row and its draft's (0: no queue), of all with the longest cursor's rows
  int32_t draw_chunk, draw_per_row, draw_ctas;   // vectors of a chunk of the draw, chunks of a row
  int32_t* status;

  // CTA b of the statistics takes chunks [b C / ctas, (b + 1) C / ctas) of all rows' C; the one
  // that has chunk x:
  __host__ __device__ int64_t chunks() const { return (int64_t)(n_rows + n_drafted) * per_row; }
  __device__ int64_t start(int b) const { return b * chunks() / ctas; }
  __device__ int owner(int64_t x) const {
    const int64_t a = (x + 1) * ctas - 1, c = chunks();
    return a >> 32 ? (int)(a / c) : (int)((uint32_t)a / (uint32_t)c);   // a 64-bit division takes ten times as long
  }
};

__device__ __forceinline__ unsigned long long lowest_first(uint32_t key, int v) {
  return (unsigned long long)key << 32 | (0xffffffffu - (uint32_t)v);
}
// Greedy: a row with a NaN, above every value's key.
constexpr unsigned long long kNanRow = ~0ull;
__device__ __forceinline__ int id_of(unsigned long long k) { return (int)(0xffffffffu - (uint32_t)k); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// What a warp has of a row, st and the largest logit among its own whole vectors, with the entries
// past the row's last one where `last`.  Greedy: returns the largest logit with its lowest id, from
// the chunk that the thread first met it in (of kStride threads); the threads that have the warp's
// read it again.  nan: the thread met one.
template <typename T, bool kGreedy, int kStride>
__device__ __forceinline__ unsigned long long warp_total(const VerifyParams& p, const T* x, float c2, bool last, float top, int top_chunk, bool nan, Stat& st) {
  constexpr int E = Vec<T>::E;
  const int tid = threadIdx.x, nv = p.V / E;
  int top_id = -1;
  if (kGreedy) {
    float all = top;
#pragma unroll
    for (int o = 16; o; o >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
    if (top_chunk >= 0 && top == all) {
      const int v = top_chunk * p.per_chunk + tid, end = min((top_chunk + 1) * p.per_chunk, nv);
      uint4 w[kPer];
#pragma unroll
      for (int q = 0; q < kPer; q++) w[q] = v + q * kStride < end ? reinterpret_cast<const uint4*>(x)[v + q * kStride] : Raw<T>::masked();
#pragma unroll
      for (int q = kPer - 1; q >= 0; q--) {
        float f[E];
        Vec<T>::cvt(w[q], f);
#pragma unroll
        for (int e = E - 1; e >= 0; e--)
          if (f[e] == top) top_id = (v + q * kStride) * E + e;
      }
    }
    __syncwarp();
  }
  if (last && tid < p.V - nv * E) {
    const int i = nv * E + tid;
    const float v = Vec<T>::get(x + i);
    if (v > st.m) st.rebase(v, c2);
    st.add(v, c2);
    if (kGreedy && v > top) top = v, top_id = i;
    nan |= v != v;
  }
  warp_merge(st, c2);
  return kGreedy ? warp_max(nan ? kNanRow : top_id >= 0 ? lowest_first(order_key(top), top_id) : 0) : 0;
}

// Softmax statistics (greedy: and the largest logits) of all rows that are needed: each CTA takes
// an equal run of chunks of up to 32 KB, over the rows' ends, and writes what it has of a row.
// The next chunk's loads are under way while one is summed or a row's sums are joined: 64 to 128
// KB an SM.  Bound by HBM.
template <typename T, bool kGreedy>
__global__ void __launch_bounds__(kThreads, kHeld) k_verify_stats(const __grid_constant__ VerifyParams p) {
  constexpr int E = Vec<T>::E;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ Stat part_st[2][kThreads / 32];
  __shared__ unsigned long long part_top[2][kThreads / 32];
  launch_dependents();
  const int nv = p.V / E;
  const int64_t x0 = p.start(blockIdx.x), x1 = p.start(blockIdx.x + 1);
  if (x0 >= x1) return;
  int row = (int)(x0 / p.per_row), chunk = (int)(x0 - (int64_t)row * p.per_row);
  auto data = [&](int r) -> const T* {
    if (r < p.n_rows) return static_cast<const T*>(p.x) + r * p.ld;
    return static_cast<const T*>(p.y) + (int64_t)(p.drafted[r - p.n_rows] - p.first) * p.yld;
  };
  const T* x = data(row);
  wait_for_predecessor();
  if (!kGreedy)
    for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < p.n_cur; i += (int64_t)p.ctas * kThreads) p.drawn[i] = 0, p.done[i] = 0;
  uint4 w[kPer], ahead[kPer];
  auto fetch = [&](const T* from, int ch) {
    const int v = ch * p.per_chunk + tid, end = min((ch + 1) * p.per_chunk, nv);
#pragma unroll
    for (int q = 0; q < kPer; q++)
      ahead[q] = v + q * kThreads < end ? __ldcs(reinterpret_cast<const uint4*>(from) + v + q * kThreads) : Raw<T>::masked();
  };
  fetch(x, chunk);
  int turn = 0;
  for (int64_t at = x0; at < x1; turn ^= 1) {
    // the chunks of this row that are this CTA's
    const int end = (int)min((int64_t)p.per_row, chunk + (x1 - at));
    const float c2 = (row < p.n_rows ? p.c : p.cy) * kLog2e;
    const T* next_x = at + (end - chunk) < x1 ? data(row + 1) : x;
    StageStat<T, false> ss;
    ss.init();
    float top = -INFINITY;     // largest logit so far, and (greedy) the first chunk that has it
    int top_chunk = -1;
    bool nan = false;          // (greedy) met one
    for (int ch = chunk; ch < end; ch++) {
#pragma unroll
      for (int q = 0; q < kPer; q++) w[q] = ahead[q];
      if (ch + 1 < end) fetch(x, ch + 1);
      else if (at + (end - chunk) < x1) fetch(next_x, 0);
      const float mx = Raw<T>::template max<kGreedy>(w);
      if (kGreedy && mx > top) top_chunk = ch;
      if (kGreedy) nan |= mx != mx;
      top = fmaxf(top, mx);
      ss.add(w, INT_MAX, mx, c2);
    }
    Stat st = ss.total(top, c2);
    const unsigned long long best = warp_total<T, kGreedy, kThreads>(p, x, c2, end == p.per_row, top, top_chunk, nan, st);
    if (lane == 0) part_st[turn][warp] = st, part_top[turn][warp] = best;
    __syncthreads();   // the arrays of the turn before are read by then
    if (warp == 0) {
      st.init();
      if (lane < kThreads / 32) st = part_st[turn][lane];
      warp_merge(st, c2);
      const unsigned long long all = kGreedy ? warp_max(lane < kThreads / 32 ? part_top[turn][lane] : 0) : 0;
      if (lane == 0) {
        const int64_t o = (int64_t)row * p.slots + (int)blockIdx.x - p.owner((int64_t)row * p.per_row);
        p.stat[o] = make_float2(st.m, st.s);
        if (kGreedy) p.best[o] = all;
      }
    }
    at += end - chunk;
    row++, chunk = 0, x = next_x;
  }
}

// ln p of a logit of a row with largest logit st.x and ln S = st.y (-inf, -inf: no logit above -inf)
__device__ __forceinline__ float log_p(float x, float2 st, float c) { return st.x == -INFINITY ? -INFINITY : (x - st.x) * c - st.y; }

// (x - m) c in two parts, to some 2^-46 of it: the difference and the product with their errors.
__device__ __forceinline__ float2 scaled_difference(float x, float m, float c) {
  const float d = __fsub_rn(x, m), b = __fsub_rn(d, x);
  const float err = __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(m, b));
  const float h = __fmul_rn(d, c);
  return make_float2(h, fmaf(err, c, fmaf(d, c, -h)));
}
// p / q = e^(ex - ey) sy / sx, ex and ey such differences: the difference of two fp32 logarithms at
// -100 would leave 1e-5 of it.
__device__ __forceinline__ float ratio(float2 ex, float sx, float2 ey, float sy) {
  const float h = __fsub_rn(ex.x, ey.x), b = __fsub_rn(h, ex.x);
  const float err = __fsub_rn(__fsub_rn(ex.x, __fsub_rn(h, b)), __fadd_rn(ey.x, b));
  const float l = err + (ex.y - ey.y);
  return expf(h) * (1.f + l) * (sy / sx);
}

// Slots of row t of the statistics that are written.
__device__ __forceinline__ int slots_of(const VerifyParams& p, int t) {
  return p.parts ? 2 : p.owner((int64_t)(t + 1) * p.per_row - 1) - p.owner((int64_t)t * p.per_row) + 1;
}
// One warp: (m, ln S) of row t of the statistics; sum: S.
__device__ __forceinline__ float2 row_stat(const VerifyParams& p, int t, float c, float& sum) {
  const int lane = threadIdx.x & 31, n = slots_of(p, t);
  const float c2 = c * kLog2e;
  Stat st;
  st.init();
  for (int i = lane; i < n; i += 32) {
    const float2 s = __ldcg(&p.stat[(int64_t)t * p.slots + i]);   // may be of another CTA of this kernel
    st.merge(s.x, s.y, 0.f, c2);
  }
  warp_merge(st, c2);
  sum = st.s;
  return st.s == 0.f ? make_float2(-INFINITY, -INFINITY) : make_float2(st.m, logf(st.s));
}
// One warp: the largest logit of a target's row (0: none above -inf).
__device__ __forceinline__ unsigned long long row_best(const VerifyParams& p, int t) {
  const int lane = threadIdx.x & 31, n = slots_of(p, t);
  unsigned long long b = 0;
  for (int i = lane; i < n; i += 32) b = max(b, __ldcg(&p.best[(int64_t)t * p.slots + i]));
  return warp_max(b);
}

// p = softmax of logits, two at a time: 2^(d hi + (d lo - log2 S)), d = x - m, hi + lo = c log2 e to
// some 48 bits: the race compares probabilities of tokens, and one rounding of d c log2 e would be
// 2^-24 of it.  hi is rounded down and lo positive, so that a masked entry's terms are both -inf.
// A row without a logit above -inf gives NaN, which wins no race.
struct Prob {
  f2 minus_m, hi, lo, minus_l2;
  __device__ __forceinline__ void set(float2 st, float h, float l) {
    minus_m = pack2(-st.x, -st.x), hi = pack2(h, h), lo = pack2(l, l);
    minus_l2 = pack2(-st.y * kLog2e, -st.y * kLog2e);
  }
  __device__ __forceinline__ f2 operator()(f2 x) const {
    const f2 d = add2(x, minus_m);
    float a, b;
    unpack2(fma2(d, hi, fma2(d, lo, minus_l2)), a, b);
    return pack2(ex2f(a), ex2f(b));
  }
};

// The race of one row: the largest w / e of this thread's entries and the lowest id that has it.
template <typename T>
struct Race {
  static constexpr int E = Vec<T>::E;
  Prob pp, pq;
  int out;          // id left out, or -1
  float top;
  int id;
  __device__ __forceinline__ void start(const Decision& d, const VerifyParams& p) {
    pp.set(d.st, p.hi[0], p.lo[0]);
    pq.set(d.y_st, p.hi[1], p.lo[1]);
    out = d.out, top = 0.f, id = 0;
  }
  // E entries from id v on; s: their w / e
  __device__ __forceinline__ void take(float (&s)[E], int v) {
    if ((uint32_t)(out - v) < (uint32_t)E) {
#pragma unroll
      for (int k = 0; k < E; k++)
        if (v + k == out) s[k] = 0.f;
    }
    float m = s[0];
#pragma unroll
    for (int k = 1; k < E; k++) m = fmaxf(m, s[k]);
    if (m > top) {   // rare after the first few
      top = m;
#pragma unroll
      for (int k = E - 1; k >= 0; k--)
        if (s[k] == m) id = v + k;
    }
  }
  template <bool kSub>
  __device__ __forceinline__ void vec(const uint4& x, const uint4& y, const float4 (&er)[E / 4], int v) {
    float s[E];
#pragma unroll
    for (int k = 0; k < E / 2; k++) {
      f2 w = pp(Raw<T>::pair(x, k));
      if (kSub) {
        float a, b;
        unpack2(pq(Raw<T>::pair(y, k)), a, b);
        w = add2(w, pack2(-a, -b));
      }
      const float4 f = er[k / 2];
      float i0, i1;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i0) : "f"(k & 1 ? f.z : f.x));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i1) : "f"(k & 1 ? f.w : f.y));
      unpack2(mul2(w, pack2(i0, i1)), s[2 * k], s[2 * k + 1]);
    }
    take(s, v);
  }
  // entry v of the row, past the last whole vector
  __device__ __forceinline__ void tail(const T* x, const T* y, const float* e, int v) {
    float s[E], w, unused, q = 0.f, i;
    unpack2(pp(pack2(Vec<T>::get(x + v), 0.f)), w, unused);
    if (y) unpack2(pq(pack2(Vec<T>::get(y + v), 0.f)), q, unused);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(i) : "f"(e[v]));
    s[0] = v == out ? 0.f : (w - q) * i;
    if (s[0] > top) top = s[0], id = v;
  }
  __device__ __forceinline__ unsigned long long key() const { return top > 0.f ? lowest_first(__float_as_uint(top), id) : 0; }
};

// One warp: row r against the draft of the row after it (draft: there is one), with probability a;
// statistics of the draft's row: y0 + r.  Returns whether it is accepted; d: the next token's
// distribution if the cursor's drafts end here, but d.acc.
template <typename T, bool kGreedy>
__device__ __forceinline__ bool weigh(const VerifyParams& p, int r, int y0, bool draft, Decision& d, float& a) {
  const T *x = static_cast<const T*>(p.x), *y = static_cast<const T*>(p.y);
  const int row = p.first + r + 1, id = draft ? p.ids[row] : -1;
  const bool known = id >= 0 && id < p.V;
  d.row = r, d.y_row = draft && y ? r : -1, d.out = draft && !y ? id : -1;
  bool taken;
  float sx, sy = 1.f;
  a = 0.f;
  if (kGreedy) {
    const unsigned long long b = row_best(p, r);
    d.out = b && b != kNanRow ? id_of(b) : -1;
    taken = known && d.out == id;
    a = taken;
    d.st = row_stat(p, r, p.c, sx);
  } else {
    const float lx = known ? Vec<T>::get(x + r * p.ld + id) : 0.f, ly = known && y ? Vec<T>::get(y + r * p.yld + id) : 0.f;
    const float u = draft ? p.u[row] : 0.f;
    d.st = row_stat(p, r, p.c, sx);
    d.y_st = draft && y ? row_stat(p, y0 + r, p.cy, sy) : make_float2(0.f, 0.f);
    if (d.y_st.x == -INFINITY) d.y_row = -1;   // a draft of nothing takes nothing off
    const float lp = log_p(lx, d.st, p.c), lq = y ? log_p(ly, d.y_st, p.cy) : 0.f;
    if (known && lq == lq && lp >= kLogZero) {   // not where one is NaN
      const float q = lq < kLogZero ? 1.f
                                      : ratio(scaled_difference(lx, d.st.x, p.c), sx,
                                              y ? scaled_difference(ly, d.y_st.x, p.cy) : make_float2(0.f, 0.f), sy);
      a = q >= 1.f ? 1.f : q;
    }
    taken = u < a;
  }
  return __shfl_sync(0xffffffffu, taken, 0);
}

// What k_verify_queue counts in, and the draw.
__global__ void __launch_bounds__(256) k_verify_clear(const __grid_constant__ VerifyParams p) {
  launch_dependents();
  wait_for_predecessor();
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < p.n_cur) p.rejected[i] = kNone, p.drawn[i] = 0, p.done[i] = 0;
  if (i < p.n_rows) p.parts_done[i] = 0;
  if (i == 0) *p.ticket = p.ctas;
}

// Unit u: cursor, its row j, half of the target's row (half < 2) or of the draft's.
struct Unit {
  int i, j, half;
  __device__ __forceinline__ Unit(const VerifyParams& p, int u) {
    const int of_row = p.n_cur * p.parts;
    j = u / of_row, i = (u - j * of_row) / p.parts, half = (u - j * of_row) % p.parts;
  }
};

// The statistics where there are many cursors: what a cursor has behind its first rejected draft
// need not be read.  Units of half a row, the cursors' first rows first, are handed out by a
// counter; when those of a row and of its draft's distribution are summed, the draft is judged, and
// the cursor's later units are passed over.  A CTA: 15 warps sum, the next chunk's loads under way;
// one in control takes the units, joins the warps' results and judges, beside them.  Bound by HBM,
// with 60 KB an SM under way where k_verify_stats has 64 (512 threads that sum and one warp more
// leave 56 registers: 145 us where 137), and by what is taken before its cursor is judged.
template <typename T, bool kGreedy>
__global__ void __launch_bounds__(kThreads, kHeld) k_verify_queue(const __grid_constant__ VerifyParams p) {
  constexpr int E = Vec<T>::E, kWarps = kSummers / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ Stat part_st[kAhead][kWarps];
  __shared__ unsigned long long part_top[kAhead][kWarps];
  __shared__ uint64_t given[kAhead], summed[kAhead];
  __shared__ int s_unit[kAhead];   // -1: no more
  launch_dependents();
  if (tid == 0) {
    for (int k = 0; k < kAhead; k++) tc::mbar_init(&given[k], 1), tc::mbar_init(&summed[k], kWarps);
    tc::fence_mbar_init();
  }
  __syncthreads();
  wait_for_predecessor();
  if (warp == kWarps) {
    // the first unit from u on that has something to sum, or -1
    auto take = [&](int u) {
      int at = -1;
      if (lane == 0)
        for (; u < p.units; u = atomicAdd(p.ticket, 1)) {
          const Unit w(p, u);
          const int n = p.row0[w.i + 1] - p.row0[w.i];
          if (w.j < n - (w.half >= 2) && w.j <= *(volatile int32_t*)&p.rejected[w.i]) {
            at = u;
            break;
          }
        }
      return __shfl_sync(0xffffffffu, at, 0);
    };
    auto next = [&] { return take(lane == 0 ? atomicAdd(p.ticket, 1) : 0); };
    auto give = [&](int k, int u) {
      if (lane == 0) {
        s_unit[k] = u;
        tc::mbar_arrive(&given[k]);
      }
    };
    int unit[kAhead];
    unit[0] = take(blockIdx.x);
    give(0, unit[0]);
    unit[1] = unit[0] < 0 ? -1 : next();
    give(1, unit[1]);
    for (int k = 0;; k++) {
      const int b = k & 1, u = b ? unit[1] : unit[0];
      if (u < 0 || !warp_wait(&summed[b], (k >> 1) & 1, p.status)) return;
      const Unit w(p, u);
      const int r0 = p.row0[w.i] - p.first, n = p.row0[w.i + 1] - p.row0[w.i], y0 = p.n_rows - (p.live[w.i] - p.live0);
      const float c2 = (w.half < 2 ? p.c : p.cy) * kLog2e;
      Stat st;
      st.init();
      if (lane < kWarps) st = part_st[b][lane];
      unsigned long long best = kGreedy && lane < kWarps ? part_top[b][lane] : 0;
      __syncwarp();
      const int after = (b ? unit[0] : unit[1]) < 0 ? -1 : next();
      (b ? unit[1] : unit[0]) = after;
      give(b, after);
      warp_merge(st, c2);
      if (kGreedy) best = warp_max(best);
      const int r = r0 + w.j, t = w.half < 2 ? r : y0 + r;
      int before = 0;
      if (lane == 0) {
        p.stat[(int64_t)t * 2 + (w.half & 1)] = make_float2(st.m, st.s);
        if (kGreedy) p.best[(int64_t)t * 2 + (w.half & 1)] = best;
        __threadfence();
        if (w.j + 1 < n) before = atomicAdd(&p.parts_done[r], 1);
        __threadfence();
      }
      before = __shfl_sync(0xffffffffu, before, 0);
      __syncwarp();
      if (w.j + 1 < n && before == p.parts - 1) {
        Decision d;
        float a;
        if (!weigh<T, kGreedy>(p, r, y0, true, d, a) && lane == 0) atomicMin(&p.rejected[w.i], w.j);
      }
      __syncwarp();
    }
  }
  const int nv = p.V / E;
  uint4 w[kPer], ahead[kPer];
  struct Row {
    const T* x;
    float c2;
    int from, to;   // chunks
  };
  auto row_of = [&](int u) {
    const Unit w(p, u);
    const int r = p.row0[w.i] - p.first + w.j, h = w.half & 1;
    Row o;
    o.x = w.half < 2 ? static_cast<const T*>(p.x) + r * p.ld : static_cast<const T*>(p.y) + r * p.yld;
    o.c2 = (w.half < 2 ? p.c : p.cy) * kLog2e;
    o.from = h ? p.per_row / 2 : 0, o.to = h ? p.per_row : p.per_row / 2;
    return o;
  };
  auto fetch = [&](const T* from, int ch) {
    const int v = ch * p.per_chunk + tid, end = min((ch + 1) * p.per_chunk, nv);
#pragma unroll
    for (int q = 0; q < kPer; q++)
      ahead[q] = v + q * kSummers < end ? __ldcs(reinterpret_cast<const uint4*>(from) + v + q * kSummers) : Raw<T>::masked();
  };
  if (!warp_wait(&given[0], 0, p.status) || s_unit[0] < 0) return;
  Row row = row_of(s_unit[0]), next = row;
  fetch(row.x, row.from);
  for (int k = 0;; k++) {
    const int b = k & 1;
    bool more = false;
    StageStat<T, false> ss;
    ss.init();
    float top = -INFINITY;
    int top_chunk = -1;
    bool nan = false;          // (greedy) met one
    for (int ch = row.from; ch < row.to; ch++) {
#pragma unroll
      for (int q = 0; q < kPer; q++) w[q] = ahead[q];
      if (ch + 1 < row.to) fetch(row.x, ch + 1);
      else {
        if (!warp_wait(&given[b ^ 1], ((k + 1) >> 1) & 1, p.status)) return;
        const int u = s_unit[b ^ 1];
        more = u >= 0;
        if (more) {
          next = row_of(u);
          fetch(next.x, next.from);
        }
      }
      const float mx = Raw<T>::template max<kGreedy>(w);
      if (kGreedy && mx > top) top_chunk = ch;
      if (kGreedy) nan |= mx != mx;
      top = fmaxf(top, mx);
      ss.add(w, INT_MAX, mx, row.c2);
    }
    Stat st = ss.total(top, row.c2);
    const unsigned long long best = warp_total<T, kGreedy, kSummers>(p, row.x, row.c2, row.to == p.per_row, top, top_chunk, nan, st);
    if (lane == 0) {
      part_st[b][warp] = st;
      if (kGreedy) part_top[b][warp] = best;
      tc::mbar_arrive(&summed[b]);
    }
    if (!more) return;
    row = next;
  }
}

// One warp's share of a cursor's decision: its rows j = w, w + step, ..., of which all but the last
// lead to a draft.  *acc: the first rejected draft so far (n - 1: none); dec: what this warp would
// decide for the last row that it looked at; writes: whether accept_p is this CTA's to write.  A
// chain of dependent loads: bound by latency.
template <typename T, bool kGreedy>
__device__ __forceinline__ void judge(const VerifyParams& p, int i, int w, int step, int* acc, Decision* dec, bool writes) {
  const int lane = threadIdx.x & 31;
  const int r0 = p.row0[i] - p.first, n = p.row0[i + 1] - p.row0[i];
  const int y0 = p.n_rows - (p.live[i] - p.live0);   // statistics of the draft's row r: y0 + r
  for (int j = w;; j += step) {
    // one reading a warp: lanes that read it apart could part here, before the shuffles of all 32
    const int limit = __shfl_sync(0xffffffffu, *(volatile int*)acc, 0);
    if (j >= n || j > limit) break;
    const int r = r0 + j, row = p.first + r + 1;   // row: of the plan, the draft's (j < n - 1)
    const bool draft = j + 1 < n;
    Decision d;
    float a;
    const bool taken = weigh<T, kGreedy>(p, r, y0, draft, d, a);
    d.acc = j;
    if (lane == 0) {
      *dec = d;
      if (draft && writes && p.accept_p) p.accept_p[row] = a;
    }
    if (draft && !taken) {
      if (lane == 0) atomicMin(acc, j);
      break;   // what comes after it does not count
    }
  }
  __syncwarp();
}
// The cursor's row, from 0 on, that its drafts end at for all that is known.
__device__ __forceinline__ int drafts_to_judge(const VerifyParams& p, int i) {
  const int last = p.row0[i + 1] - p.row0[i] - 1;
  return p.parts ? min(last, p.rejected[i]) : last;
}
// Threads t of `step`, when a cursor is judged: accept_p of the first row and behind the first
// rejected draft is 0; a rejected id out of range is an error.
__device__ __forceinline__ void judged(const VerifyParams& p, int i, int acc, int t, int step) {
  const int a = p.row0[i], n = p.row0[i + 1] - a;
  if (p.accept_p) {
    if (t == 0 && n > 0) p.accept_p[a] = 0.f;
    for (int j = acc + 2 + t; j < n; j += step) p.accept_p[a + j] = 0.f;
  }
  if (t == 0 && acc + 1 < n) {
    const int id = p.ids[a + acc + 1];
    if (id < 0 || id >= p.V) atomicExch(p.status, OCTO_EINVAL);
  }
}
// a cursor without rows, or whose next token is `id`
template <typename T>
__device__ __forceinline__ void result(const VerifyParams& p, int i, int acc, int id, int row, float2 st) {
  p.n_accept[i] = acc, p.next_id[i] = id;
  if (p.next_logp) p.next_logp[i] = id < 0 ? -INFINITY : log_p(Vec<T>::get(static_cast<const T*>(p.x) + row * p.ld + id), st, p.c);
}

// Greedy: a CTA a cursor, a warp a row.
template <typename T>
__global__ void __launch_bounds__(kDecide) k_verify_decide(const __grid_constant__ VerifyParams p) {
  constexpr int kWarps = kDecide / 32;
  const int tid = threadIdx.x, i = blockIdx.x;
  __shared__ int s_acc;
  __shared__ Decision s_dec[kWarps];
  launch_dependents();
  wait_for_predecessor();
  if (tid == 0) s_acc = drafts_to_judge(p, i);
  __syncthreads();
  judge<T, true>(p, i, tid / 32, kWarps, &s_acc, &s_dec[tid / 32], true);
  __syncthreads();
  const int acc = s_acc;   // its warp looked at row acc last
  judged(p, i, acc, tid, kDecide);
  if (tid) return;
  if (acc < 0) result<T>(p, i, 0, -1, 0, make_float2(0.f, 0.f));
  else result<T>(p, i, acc, s_dec[acc % kWarps].out, s_dec[acc % kWarps].row, s_dec[acc % kWarps].st);
}

// The draw of the cursors' next tokens: one CTA an SM, each with an equal run of chunks over the
// cursors' ends.  First the CTA's cursors are judged, up to 16 at a time, a warp a row; a cursor of
// several CTAs is judged in each, which takes no longer than a kernel of its own before this one.
// Then one thread copies the chunks of logits, the draft's and the noise into a ring (bulk copies,
// 190 KB under way); 16 warps race over them, a vector a thread, and take what they have of a
// cursor to its best score; the last CTA of a cursor writes its results.  Bound by HBM.
template <typename T>
struct DrawShape {
  static constexpr int E = Vec<T>::E;
  static constexpr int kVec = 512;                               // vectors of a chunk, at most
  static constexpr int kStage = kVec * (32 + 4 * E);             // logits, draft, noise
  static constexpr int kStages = 192 * 1024 / kStage;
  static constexpr int kConsumers = 512, kBlock = kConsumers + 32;
  static constexpr int kSmem = kStages * kStage + 256;
};

template <typename T>
__global__ void __launch_bounds__(DrawShape<T>::kBlock, 1) k_verify_draw(const __grid_constant__ VerifyParams p) {
  using S = DrawShape<T>;
  constexpr int E = S::E, kWarps = S::kConsumers / 32;
  extern __shared__ __align__(128) uint8_t sm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::kStages * S::kStage);
  uint64_t* empty = full + S::kStages;
  __shared__ unsigned long long s_best[2], s_all, s_own;
  __shared__ bool s_last;
  __shared__ int s_acc[kWarps];
  __shared__ Decision s_dec[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  launch_dependents();
  if (tid == 0) {
    for (int k = 0; k < S::kStages; k++) tc::mbar_init(&full[k], 1), tc::mbar_init(&empty[k], kWarps);
    tc::fence_mbar_init();
    s_best[0] = s_best[1] = 0;
  }
  const int nv = p.V / E;
  const int64_t C = (int64_t)p.n_cur * p.draw_per_row;
  const int64_t x0 = blockIdx.x * C / p.draw_ctas, x1 = (blockIdx.x + 1) * C / p.draw_ctas;
  auto owner = [&](int64_t x) { return (int)(((x + 1) * p.draw_ctas - 1) / C); };
  const int first = (int)(x0 / p.draw_per_row), last = (int)((x1 - 1) / p.draw_per_row);
  auto sync = [] { __syncwarp(), tc::named_bar_sync(1, S::kConsumers); };
  int st = 0, issued = 0, turn = 0;
  uint32_t round = 0;
  bool ok = true;
  for (int i0 = first; i0 <= last; i0 += kWarps) {
    const int i1 = min(i0 + kWarps, last + 1), each = kWarps / (i1 - i0);   // cursors [i0, i1), warps for each
    if (i0 == first) wait_for_predecessor();
    if (tid < i1 - i0) s_acc[tid] = drafts_to_judge(p, i0 + tid);
    __syncthreads();
    auto first_owner = [&](int i) { return (int64_t)i * p.draw_per_row >= x0; };
    if (warp < each * (i1 - i0)) judge<T, false>(p, i0 + warp / each, warp % each, each, &s_acc[warp / each], &s_dec[warp], first_owner(i0 + warp / each));
    __syncthreads();
    // the chunks of cursor i that are this CTA's: [chunk0, chunk1)
    auto chunk0 = [&](int i) { return (int)max((int64_t)0, x0 - (int64_t)i * p.draw_per_row); };
    auto chunk1 = [&](int i) { return (int)min((int64_t)p.draw_per_row, x1 - (int64_t)i * p.draw_per_row); };
    for (int i = i0; i < i1; i++) {
      const int acc = s_acc[i - i0];   // its warp looked at row acc last
      if (acc < 0) continue;
      const Decision d = s_dec[(i - i0) * each + acc % each];
      const T* x = static_cast<const T*>(p.x) + d.row * p.ld;
      const T* y = d.y_row >= 0 ? static_cast<const T*>(p.y) + d.y_row * p.yld : nullptr;
      const float* e = p.noise + i * p.eld;
      if (warp == kWarps) {
        if (lane) continue;
        for (int ch = chunk0(i); ch < chunk1(i); ch++) {
          const int v0 = ch * p.draw_chunk, cnt = min(p.draw_chunk, nv - v0);
          if (cnt <= 0) break;
          if (ok && issued >= S::kStages) ok = ring_wait(&empty[st], round ^ 1, p.status);
          if (!ok) break;
          uint8_t* dst = sm + st * S::kStage;
          tc::mbar_expect_tx(&full[st], (uint32_t)cnt * (y ? 32 + 4 * E : 16 + 4 * E));
          bulk_load(dst, x + (int64_t)v0 * E, cnt * 16, &full[st], true);
          if (y) bulk_load(dst + S::kVec * 16, y + (int64_t)v0 * E, cnt * 16, &full[st], true);
          bulk_load(dst + S::kVec * 32, e + (int64_t)v0 * E, cnt * 4 * E, &full[st], true);
          issued++;
          if (++st == S::kStages) st = 0, round ^= 1;
        }
        continue;
      }
      Race<T> race;
      race.start(d, p);
      const int end = chunk1(i);
      for (int k = chunk0(i); k < end; k++) {
        const int v0 = k * p.draw_chunk, cnt = min(p.draw_chunk, nv - v0);
        if (cnt <= 0) break;
        if (ok) ok = warp_wait(&full[st], round, p.status);
        if (ok && tid < cnt) {
          const uint8_t* src = sm + st * S::kStage;
          const uint4 xr = reinterpret_cast<const uint4*>(src)[tid];
          float4 er[E / 4];
#pragma unroll
          for (int q = 0; q < E / 4; q++) er[q] = reinterpret_cast<const float4*>(src + S::kVec * 32)[tid * (E / 4) + q];
          if (y) race.template vec<true>(xr, reinterpret_cast<const uint4*>(src + S::kVec * 16)[tid], er, (v0 + tid) * E);
          else race.template vec<false>(xr, xr, er, (v0 + tid) * E);
        }
        give_back(&empty[st], race.top);
        if (++st == S::kStages) st = 0, round ^= 1;
      }
      if (end == p.draw_per_row && tid < p.V - nv * E) race.tail(x, y, e, nv * E + tid);
      unsigned long long best = warp_max(race.key());
      if (lane == 0 && best) atomicMax(&s_best[turn], best);
      sync();
      turn ^= 1;
      if (tid == 0) {
        best = s_best[turn ^ 1];
        s_best[turn] = 0;   // of the cursor before, read by then
        if (best) atomicMax(&p.drawn[i], best);
        const int n = owner((int64_t)(i + 1) * p.draw_per_row - 1) - owner((int64_t)i * p.draw_per_row) + 1;
        __threadfence();
        s_last = atomicAdd(&p.done[i], 1) == n - 1;
        __threadfence();
        s_all = atomicMax(&p.drawn[i], 0ull), s_own = 0;
      }
      sync();
      if (!s_last) continue;
      best = s_all;
      if (best == 0 && (d.y_row >= 0 || d.out >= 0)) {
        // nothing left of p: the target's own
        race.start(d, p);
        race.out = -1;
        for (int v = tid; v < nv; v += S::kConsumers) {
          const uint4 xr = reinterpret_cast<const uint4*>(x)[v];
          float4 er[E / 4];
#pragma unroll
          for (int q = 0; q < E / 4; q++) er[q] = reinterpret_cast<const float4*>(e)[(int64_t)v * (E / 4) + q];
          race.template vec<false>(xr, xr, er, v * E);
        }
        if (tid < p.V - nv * E) race.tail(x, nullptr, e, nv * E + tid);
        best = warp_max(race.key());
        if (lane == 0 && best) atomicMax(&s_own, best);
        sync();
        best = s_own;
      }
      if (tid == 0) result<T>(p, i, d.acc, best ? id_of(best) : -1, d.row, d.st);
      sync();   // the shared results are read before the next cursor's
    }
    // what is left to write of the cursors that begin in this CTA
    if (warp < kWarps)
      for (int i = i0 + warp; i < i1; i += kWarps)
        if (first_owner(i)) {
          judged(p, i, s_acc[i - i0], lane, 32);
          if (s_acc[i - i0] < 0 && lane == 0) result<T>(p, i, 0, -1, 0, make_float2(0.f, 0.f));
        }
    __syncwarp();
    __syncthreads();   // the decisions are read before the next ones
  }
  // what was started has landed before the CTA ends
  if (tid == S::kConsumers)
    for (int k = max(0, issued - S::kStages); k < issued; k++) ring_wait(&full[k % S::kStages], (k / S::kStages) & 1, p.status);
}

int held_ctas() { return kHeld * std::max(1, sm_count()); }
// (row, slot) pairs of the statistics: rows (ctas / rows + 2) at most
size_t stat_count(int64_t rows) { return (size_t)(held_ctas() + 4 * rows); }

struct Layout {   // of the workspace
  size_t best, drawn, done, rejected, parts_done, bytes;
  Layout(int64_t rows, int64_t n_cur) {
    best = align_up(stat_count(rows) * sizeof(float2), 256);
    drawn = best + align_up(stat_count(rows) * 8, 256);
    done = drawn + align_up((size_t)n_cur * 8, 256);
    rejected = done + (size_t)n_cur * 4;
    parts_done = rejected + (size_t)n_cur * 4;
    bytes = parts_done + (size_t)rows * 4 + 4;
  }
};

// The queue takes rows of four chunks at least (its units are half a row), cursors enough that a
// row's units come three units' times after those of the row before, drafts enough, and cursors of
// alike many rows, for the longest one's count of each is handed out.  256 cursors of five rows,
// 0.5, 1.3 and 4 of four drafts accepted: 126, 137 and 163 us, else 161, 161 and 152; 512 cursors
// 207, 229 and 306, else 309, 307 and 289; 512 greedily, without drafts' distributions, 1.8 and 4
// accepted: 99 and 142, else 144.  256 cursors of three rows, 0.4, 1 and 2 of two accepted: 112, 112
// and 115, else 115, 113 and 107, so four rows at least.  (Units of a quarter: 256 cursors of five
// rows 136, 150 and 184.)
constexpr int kQueueChunks = 4;
template <typename T, bool kGreedy>
int run(VerifyParams& p, cudaStream_t s) {
  const int nv = p.V / Vec<T>::E;
  p.per_row = std::max(1, (nv + kChunk - 1) / kChunk);
  p.per_chunk = (nv + p.per_row - 1) / p.per_row;
  const int64_t rows = (int64_t)p.n_rows + p.n_drafted;
  if (rows > INT32_MAX / 4) return OCTO_EINVAL;
  p.parts = 0;
  const int32_t per_row = (nv + kPer * kSummers - 1) / (kPer * kSummers), parts = p.y ? 4 : 2;
  // (the counter's steps past the end fit)
  if (per_row >= kQueueChunks && (int64_t)p.n_cur * parts >= 3 * held_ctas() && p.longest > 3 &&
      (int64_t)p.n_cur * p.longest <= 2LL * p.n_rows && p.n_rows < (1 << 26)) {
    p.parts = parts;
    p.units = p.n_cur * p.longest * parts;
    p.per_row = per_row;
    p.per_chunk = (nv + per_row - 1) / per_row;
    p.ctas = held_ctas();
    p.slots = 2;
    if (int st = launch_overlapped((const void*)k_verify_clear, &p, (std::max(p.n_rows, p.n_cur) + 255) / 256, 256, 1, 0, s)) return st;
    if (int st = launch_overlapped((const void*)k_verify_queue<T, kGreedy>, &p, p.ctas, kThreads, 1, 0, s)) return st;
  } else if (rows > 0) {
    p.ctas = (int)std::min<int64_t>(held_ctas(), p.chunks());
    p.slots = (int)(p.ctas / rows + 2);
    if (int st = launch_overlapped((const void*)k_verify_stats<T, kGreedy>, &p, p.ctas, kThreads, 1, 0, s)) return st;
  }
  if (kGreedy || rows == 0) return launch_overlapped((const void*)k_verify_decide<T>, &p, p.n_cur, kDecide, 1, 0, s);
  using S = DrawShape<T>;
  p.draw_per_row = std::max(1, (nv + S::kVec - 1) / S::kVec);
  p.draw_chunk = (nv + p.draw_per_row - 1) / p.draw_per_row;
  p.draw_ctas = (int)std::min<int64_t>(std::max(1, sm_count()), (int64_t)p.n_cur * p.draw_per_row);
  if (int st = set_smem_limit((const void*)k_verify_draw<T>, S::kSmem)) return st;
  return launch_overlapped((const void*)k_verify_draw<T>, &p, p.draw_ctas, S::kBlock, 1, S::kSmem, s);
}

}  // namespace
}  // namespace octo

extern "C" {

int octo_verify_drafts_workspace_size(octo_plan_t plan, int32_t cur0, int32_t n_cur, size_t* bytes) {
  if (!plan || !plan->chunk || !bytes || cur0 < 0 || n_cur < 0 || (int64_t)cur0 + n_cur > plan->info.n_segments) return OCTO_EINVAL;
  const int64_t rows = plan->chunk->row0[cur0 + n_cur] - plan->chunk->row0[cur0];
  *bytes = octo::Layout(rows, n_cur).bytes;
  return OCTO_OK;
}

int octo_verify_drafts(octo_plan_t plan, int32_t cur0, int32_t n_cur, const void* logits, int32_t dtype, int64_t ld,
                       int32_t vocab, float inv_temp, const int32_t* ids, const void* draft_logits, int64_t draft_ld,
                       float draft_inv_temp, const float* u, const float* noise, int64_t noise_ld, int32_t* n_accept,
                       int32_t* next_id, float* next_logp, float* accept_p, void* ws, size_t ws_bytes, void* stream) {
  octo::NvtxRange nv("octo_verify_drafts");
  size_t need = 0;
  if (int st = octo_verify_drafts_workspace_size(plan, cur0, n_cur, &need)) return st;
  const int32_t first = plan->chunk->row0[cur0], n = plan->chunk->row0[cur0 + n_cur] - first;
  if (int st = octo::rows::check_rows(plan, first, n, logits, dtype, ld, vocab, inv_temp)) return st;
  const bool greedy = !u && !noise;
  if (!greedy && (!u || !noise)) return OCTO_EINVAL;
  if (draft_logits) {
    if (greedy) return OCTO_EINVAL;
    if (int st = octo::rows::check_rows(plan, first, n, draft_logits, dtype, draft_ld, vocab, draft_inv_temp)) return st;
  }
  if (noise && (noise_ld < vocab || noise_ld % 4 || ((uintptr_t)noise & 15))) return OCTO_EINVAL;
  if (n_cur > 0 && (!n_accept || !next_id)) return OCTO_EINVAL;
  if (n_cur > 0 && (!ws || ws_bytes < need || ((uintptr_t)ws & 15))) return OCTO_EINVAL;
  if (n > 0 && !ids) return OCTO_EINVAL;
  if (n_cur == 0) return OCTO_OK;
  octo::VerifyParams p;
  p.x = logits, p.y = draft_logits;
  p.ld = ld, p.yld = draft_ld, p.eld = noise_ld;
  p.V = vocab;
  p.c = inv_temp, p.cy = draft_inv_temp;
  for (int k = 0; k < 2; k++) {
    const double c2 = (double)(k ? draft_inv_temp : inv_temp) * 1.4426950408889634074;
    p.hi[k] = (float)c2;
    if (p.hi[k] > c2) p.hi[k] = std::nextafter(p.hi[k], 0.f);
    p.lo[k] = std::max((float)(c2 - p.hi[k]), FLT_MIN);
  }
  p.row0 = plan->seg_row_base + cur0;
  p.first = first;
  p.ids = ids, p.u = u, p.noise = noise;
  p.n_accept = n_accept, p.next_id = next_id, p.next_logp = next_logp, p.accept_p = accept_p;
  const octo::Layout at(n, n_cur);
  char* w = static_cast<char*>(ws);
  p.stat = reinterpret_cast<float2*>(w);
  p.best = reinterpret_cast<unsigned long long*>(w + at.best);
  p.drawn = reinterpret_cast<unsigned long long*>(w + at.drawn);
  p.done = reinterpret_cast<int32_t*>(w + at.done);
  p.rejected = reinterpret_cast<int32_t*>(w + at.rejected);
  p.parts_done = reinterpret_cast<int32_t*>(w + at.parts_done);
  p.ticket = p.parts_done + n;
  p.longest = 0;
  for (int32_t i = cur0; i < cur0 + n_cur; i++) p.longest = std::max(p.longest, plan->chunk->row0[i + 1] - plan->chunk->row0[i]);
  const std::vector<int32_t>& live = plan->chunk->live;
  p.live = plan->chunk->d_live + cur0, p.live0 = live[cur0];
  p.drafted = plan->chunk->drafted + (first - live[cur0]);
  p.n_drafted = draft_logits ? n - (live[cur0 + n_cur] - live[cur0]) : 0;
  p.n_rows = n, p.n_cur = n_cur;
  p.status = plan->pool->d_status;
  cudaStream_t s = (cudaStream_t)stream;
  plan->last_stream = s;
  if (dtype == OCTO_DTYPE_BF16)
    return greedy ? octo::run<__nv_bfloat16, true>(p, s) : octo::run<__nv_bfloat16, false>(p, s);
  return greedy ? octo::run<float, true>(p, s) : octo::run<float, false>(p, s);
}

}  // extern "C"
