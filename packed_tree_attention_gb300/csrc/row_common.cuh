// Pieces shared by the kernels that work on rows of logits (token scoring, distillation):
// 16-byte vectors of bf16 or fp32 logits, running softmax statistics, and the tokens whose
// terms a packed row feeds.
#pragma once

#include <cuda_bf16.h>
#include <float.h>
#include <math.h>

#include "internal.h"

namespace octo {
namespace rows {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kMaxSucc = 64;   // successors of one row (checked by the entry points)
constexpr int kMaxTop = 128;   // alternatives, teacher entries
// Exponents (base 2) are cut off here: 2^-1000 is 0 in fp32, and 0 * (-1000) is 0 where
// 0 * (-inf), a masked logit's term of the entropy, would be NaN.
constexpr float kCut = -1000.f;

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// maximum that keeps a NaN (fmaxf drops it, and a row with a NaN logit would look sound)
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int E = 8;
  __device__ __forceinline__ static void cvt(const uint4 w, float (&x)[E]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static uint4 pack(const float (&g)[E]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      __nv_bfloat162 b = __floats2bfloat162_rn(g[2 * i], g[2 * i + 1]);
      u[i] = *reinterpret_cast<uint32_t*>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ static float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  __device__ __forceinline__ static void put(__nv_bfloat16* p, float g) { *p = __float2bfloat16_rn(g); }
};
template <>
struct Vec<float> {
  static constexpr int E = 4;
  __device__ __forceinline__ static void cvt(const uint4 w, float (&x)[E]) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
  }
  __device__ __forceinline__ static uint4 pack(const float (&g)[E]) {
    return make_uint4(__float_as_uint(g[0]), __float_as_uint(g[1]), __float_as_uint(g[2]), __float_as_uint(g[3]));
  }
  __device__ __forceinline__ static float get(const float* p) { return *p; }
  __device__ __forceinline__ static void put(float* p, float g) { *p = g; }
};

// Running softmax statistics of the logits seen so far: m their maximum (kept finite, so
// that differences from it are never inf - inf), s = sum 2^t, a = sum 2^t t with
// t = c2 (x - m), c2 = inv_temp log2 e.  The difference is taken before the product: a
// masked logit at the type's lowest value times log2 e would overflow.  All terms of s have
// one sign and all of a the other, so ln 2 (log2 s - a / s), the entropy, cancels nothing.
struct Stat {
  float m, s, a;
  __device__ __forceinline__ void init() { m = -FLT_MAX, s = 0.f, a = 0.f; }
  // moves the reference to mn >= m: every t falls by d = c2 (mn - m)
  __device__ __forceinline__ void rebase(float mn, float c2) {
    const float d = max_nan((m - mn) * c2, kCut);
    const float f = ex2f(d);
    a = f * fmaf(d, s, a);
    s *= f;
    m = mn;
  }
  __device__ __forceinline__ void add(float x, float c2) {
    const float t = max_nan((x - m) * c2, kCut);
    const float e = ex2f(t);
    s += e;
    a = fmaf(e, t, a);
  }
  __device__ __forceinline__ void merge(float m2, float s2, float a2, float c2) {
    Stat o{m2, s2, a2};
    const float mn = fmaxf(m, m2);
    rebase(mn, c2);
    o.rebase(mn, c2);
    s += o.s;
    a += o.a;
  }
};

// Order-preserving key of a logit: unsigned order is the order of the values, +0 and -0
// equal; 0 for a NaN (never an alternative), 1 at least for a value.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if (x != x) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// The tokens whose terms row r of a plan feeds.  Pack plan: the next row of r's segment and
// the first rows of the segments that continue from r (at most kMaxSucc in all).  Decode
// plan: the cursor's next token, which has r's own index.
struct SuccTable {
  const int32_t* seg_row_base;
  const int32_t* seg_pred;
  const int32_t* ex_pred;   // extra successors, sorted by predecessor row
  const int32_t* ex_row;
  int32_t n_segs, n_rows, n_ex, is_decode;

  // One thread, a row of a pack plan: its segment's end, whether it starts a path, and its extra
  // successors ex_row[e0, e0 + n).  The row's segment is the last one whose first row is <= r
  // (empty segments before it share its first row, empty ones after it start past r).
  __device__ void locate(int r, int* end, bool* path_start, int* e0, int* n) const {
    int lo = 0, hi = n_segs - 1, a = 0, b = n_ex;
    while (lo < hi || a < b) {
      const int mid = (lo + hi + 1) >> 1, em = (a + b) >> 1;
      const bool seg = lo < hi, ex = a < b;
      const int base = seg ? seg_row_base[mid] : 0, pred = ex ? ex_pred[em] : 0;
      if (seg) {
        if (base <= r) lo = mid;
        else hi = mid - 1;
      }
      if (ex) {
        if (pred < r) a = em + 1;
        else b = em;
      }
    }
    *end = lo + 1 < n_segs ? seg_row_base[lo + 1] : n_rows;
    *path_start = r == seg_row_base[lo] && seg_pred[lo] < 0;
    *e0 = a;
    *n = 0;
    while (*n < kMaxSucc && a + *n < n_ex && ex_pred[a + *n] == r) ++*n;
  }

  // One warp: row r's successors into t; returns how many.  Each step narrows a search to a
  // 32nd, so that a call waits for one or two loads in a row and not for a binary search of them.
  __device__ int find(int r, int32_t* t) const {
    const int lane = threadIdx.x & 31;
    if (is_decode) {
      if (lane == 0) t[0] = r;
      return 1;
    }
    int lo = 0, hi = n_segs, a = 0, b = n_ex;   // the segment is in [lo, hi), the first extra in [a, b]
    for (;;) {
      const int s1 = (hi - lo + 31) / 32, s2 = max(1, (b - a + 31) / 32);
      const int i = lo + lane * s1, e = a + lane * s2;
      const int base = i < n_segs ? seg_row_base[i] : INT32_MAX, pred = e < n_ex ? ex_pred[e] : INT32_MAX;
      const int k = 31 - __clz(__ballot_sync(0xffffffffu, base <= r && i < hi));
      const uint32_t below = __ballot_sync(0xffffffffu, pred < r && e < b);
      if (s1 == 1 && s2 == 1) {
        const int after = __shfl_down_sync(0xffffffffu, base, 1);
        int end = __shfl_sync(0xffffffffu, after, k);
        if (k == 31) end = lo + 32 < n_segs ? seg_row_base[lo + 32] : n_rows;
        if (end == INT32_MAX) end = n_rows;
        int n = 0;
        if (r + 1 < end) {
          if (lane == 0) t[0] = r + 1;
          n = 1;
        }
        for (int at = a + __popc(below); n < kMaxSucc; at += 32) {
          const bool mine = at + lane < n_ex && ex_pred[at + lane] == r;
          if (mine && n + lane < kMaxSucc) t[n + lane] = ex_row[at + lane];
          const int more = __popc(__ballot_sync(0xffffffffu, mine));
          n = min(n + more, kMaxSucc);
          if (more < 32) break;
        }
        return n;
      }
      const int nlo = lo + k * s1;
      hi = min(hi, nlo + s1);
      lo = nlo;
      const int c = __popc(below);   // the first extra is past entry c - 1 and not past entry c
      b = min(b, a + c * s2);
      a = c ? a + (c - 1) * s2 + 1 : a;
      if (a > b) a = b;
    }
  }
};

inline SuccTable succ_table(const octo_plan_s* p) {
  SuccTable t;
  t.seg_row_base = p->seg_row_base;
  t.seg_pred = p->seg_pred;
  t.ex_pred = p->succ_pred;
  t.ex_row = p->succ_row;
  t.n_segs = (int32_t)p->info.n_segments;
  t.n_rows = (int32_t)p->info.n_rows;
  t.n_ex = p->n_succ_extra;
  t.is_decode = p->info.is_decode;
  return t;
}

// The arguments that every call on rows of logits has in common.
inline int check_rows(const octo_plan_s* plan, int32_t row0, int32_t n_rows, const void* logits, int32_t dtype,
                      int64_t ld, int32_t vocab, float inv_temp) {
  if (!plan) return OCTO_EINVAL;
  if (row0 < 0 || n_rows < 0 || (int64_t)row0 + n_rows > plan->info.n_rows || vocab < 1 || ld < vocab) return OCTO_EINVAL;
  if (dtype != OCTO_DTYPE_BF16 && dtype != OCTO_DTYPE_F32) return OCTO_EINVAL;
  if (!(inv_temp > 0.f) || !std::isfinite(inv_temp)) return OCTO_EINVAL;
  const size_t es = dtype == OCTO_DTYPE_BF16 ? 2 : 4;
  if (((uintptr_t)logits & 15) || ((size_t)ld * es) % 16) return OCTO_EINVAL;
  if (n_rows > 0 && !logits) return OCTO_EINVAL;
  int dev = 0;
  OCTO_CUDA(cudaGetDevice(&dev));
  return dev == plan->device ? OCTO_OK : OCTO_EINVAL;
}

}  // namespace rows
}  // namespace octo
