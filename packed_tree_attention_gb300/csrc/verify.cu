// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// With p_r = softmax(c x_r) the target's distribution after row r and q_r the draft's, the draft
// in row r + 1, token y, is accepted with probability a = min(1, p_r(y) / q_r(y)); after the
// first rejected one the next token is drawn from max(0, p_r - q_r) / sum, else from p.  A draw
// from weights w is argmax_v w_v / e_v with e_v ~ Exp(1) independent (the first of exponential
// clocks of rates w_v), so that neither a sum of the weights nor an order of them is needed.

#include <algorithm>

#include "chunk.h"
#include "row_common.cuh"
#include "row_ring.cuh"

namespace octo {
namespace {

using namespace rows;

constexpr int kStatThreads = 512;
constexpr int kPickThreads = 1024;

struct VerifyParams {
  const void *x, *y;          // target's and draft's logits
  int64_t ld, yld, eld;
  int32_t V;
  float c, cy;                // inverse temperatures
  const int32_t* row0;        // [cursors + 1] first row of the plan's cursors, from cur0 on
  int32_t first;              // row0[0]
  const int32_t* ids;
  const float *u, *noise;
  int32_t *n_accept, *next_id;
  float *next_logp, *accept_p;
  float2* stat;               // [2][rows] (m, ln S) of the target's and the draft's rows
  unsigned long long* best;   // [rows] greedy: order_key of the largest logit, ~id
  int32_t n_rows;
  int32_t* status;
};

__device__ __forceinline__ unsigned long long lowest_first(uint32_t key, int v) {
  return (unsigned long long)key << 32 | (0xffffffffu - (uint32_t)v);
}
__device__ __forceinline__ int id_of(unsigned long long k) { return (int)(0xffffffffu - (uint32_t)k); }

template <typename T, bool kGreedy>
__global__ void __launch_bounds__(kStatThreads) k_verify_stats(const __grid_constant__ VerifyParams p) {
  constexpr int E = Vec<T>::E;
  const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool draft = blockIdx.y;
  const T* x = draft ? static_cast<const T*>(p.y) + r * p.yld : static_cast<const T*>(p.x) + r * p.ld;
  const float c2 = (draft ? p.cy : p.c) * kLog2e;
  Stat st;
  st.init();
  unsigned long long best = 0;
  auto one = [&](float v, int i) {
    st.add(v, c2);
    if (kGreedy) {
      const uint32_t k = order_key(v);
      if (k > (uint32_t)(best >> 32)) best = lowest_first(k, i);
    }
  };
  for (int i = tid; i < p.V / E; i += kStatThreads) {
    float v[E];
    Vec<T>::cvt(reinterpret_cast<const uint4*>(x)[i], v);
    float mx = v[0];
#pragma unroll
    for (int e = 1; e < E; e++) mx = fmaxf(mx, v[e]);
    if (mx > st.m) st.rebase(mx, c2);
#pragma unroll
    for (int e = 0; e < E; e++) one(v[e], i * E + e);
  }
  for (int i = p.V / E * E + tid; i < p.V; i += kStatThreads) {
    const float v = Vec<T>::get(x + i);
    if (v > st.m) st.rebase(v, c2);
    one(v, i);
  }
  __shared__ Stat part[kStatThreads / 32];
  __shared__ unsigned long long top[kStatThreads / 32];
  warp_merge(st, c2);
#pragma unroll
  for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) part[warp] = st, top[warp] = best;
  __syncthreads();
  if (tid) return;
  for (int w = 1; w < kStatThreads / 32; w++) st.merge(part[w].m, part[w].s, part[w].a, c2), best = max(best, top[w]);
  // every logit -inf: the largest stayed at the start's reference, far below, and nothing summed
  const bool none = st.s == 0.f;
  p.stat[draft * p.n_rows + r] = make_float2(none ? -INFINITY : st.m, none ? -INFINITY : logf(st.s));
  if (kGreedy) p.best[r] = best;
}

__device__ __forceinline__ float log_p(float x, float2 st, float c) { return st.x == -INFINITY ? -INFINITY : (x - st.x) * c - st.y; }

// One CTA per cursor: which drafts are accepted, then the draw.
template <typename T, bool kGreedy>
__global__ void __launch_bounds__(kPickThreads) k_verify_pick(const __grid_constant__ VerifyParams p) {
  const int i = blockIdx.x, tid = threadIdx.x;
  const int r0 = p.row0[i] - p.first, n = p.row0[i + 1] - p.row0[i];
  const T *x = static_cast<const T*>(p.x), *y = static_cast<const T*>(p.y);
  __shared__ int s_acc;
  __shared__ unsigned long long s_best;
  if (n == 0) {
    if (tid == 0) {
      p.n_accept[i] = 0, p.next_id[i] = -1;
      if (p.next_logp) p.next_logp[i] = -INFINITY;
    }
    return;
  }
  if (tid == 0) {
    int acc = 0;
    bool on = true;
    if (p.accept_p) p.accept_p[p.first + r0] = 0.f;
    for (int j = 0; j + 1 < n; j++) {
      const int r = r0 + j, row = p.first + r + 1;   // row: of the plan, the draft's
      float a = 0.f;
      bool taken = false;
      if (on) {
        const int id = p.ids[row];
        if (id < 0 || id >= p.V) {
          atomicExch(p.status, OCTO_EINVAL);
        } else if (kGreedy) {
          const unsigned long long b = p.best[r];
          taken = b >> 32 && p.stat[r].x != -INFINITY && id_of(b) == id;
          a = taken;
        } else {
          const float lp = log_p(Vec<T>::get(x + r * p.ld + id), p.stat[r], p.c);
          const float lq = y ? log_p(Vec<T>::get(y + r * p.yld + id), p.stat[p.n_rows + r], p.cy) : 0.f;
          a = lp == -INFINITY ? 0.f : lp >= lq ? 1.f : expf(lp - lq);
          if (!(lp == lp) || !(lq == lq)) a = 0.f;
          taken = p.u[row] < a;
        }
      }
      if (p.accept_p) p.accept_p[row] = a;
      on = taken;
      acc += taken;
    }
    s_acc = acc;
    s_best = 0;
  }
  __syncthreads();
  const int acc = s_acc, r = r0 + acc;
  const bool rejected = acc + 1 < n;
  const float2 st = p.stat[r];
  unsigned long long best = 0;
  if (kGreedy) {
    best = st.x == -INFINITY ? 0 : p.best[r];
  } else {
    const float2 sq = rejected && y ? p.stat[p.n_rows + r] : make_float2(0.f, 0.f);
    const int out = rejected && !y ? p.ids[p.first + r + 1] : -1;
    const float* e = p.noise + i * p.eld;
    for (int pass = 0; pass < 2 && best == 0; pass++) {
      for (int v = tid; v < p.V; v += kPickThreads) {
        float w = expf(log_p(Vec<T>::get(x + r * p.ld + v), st, p.c));
        if (pass == 0) {
          if (rejected && y) w -= expf(log_p(Vec<T>::get(y + r * p.yld + v), sq, p.cy));
          if (v == out) w = 0.f;
        }
        const float s = w / e[v];
        if (s > 0.f && __float_as_uint(s) > (uint32_t)(best >> 32)) best = lowest_first(__float_as_uint(s), v);
      }
      atomicMax(&s_best, best);
      __syncthreads();
      best = s_best;
    }
  }
  if (tid) return;
  const int id = best ? id_of(best) : -1;
  p.n_accept[i] = acc;
  p.next_id[i] = id;
  if (p.next_logp) p.next_logp[i] = id < 0 ? -INFINITY : log_p(Vec<T>::get(x + r * p.ld + id), st, p.c);
}

size_t stat_bytes(int64_t rows) { return align_up((size_t)rows * 2 * sizeof(float2), 256); }

template <typename T, bool kGreedy>
int run(const VerifyParams& p, int32_t n_cur, cudaStream_t s) {
  if (p.n_rows > 0) {
    k_verify_stats<T, kGreedy><<<dim3(p.n_rows, p.y ? 2 : 1), kStatThreads, 0, s>>>(p);
    count_launch();
  }
  k_verify_pick<T, kGreedy><<<n_cur, kPickThreads, 0, s>>>(p);
  count_launch();
  return cuda_status(cudaGetLastError());
}

}  // namespace
}  // namespace octo

extern "C" {

int octo_verify_drafts_workspace_size(octo_plan_t plan, int32_t cur0, int32_t n_cur, size_t* bytes) {
  if (!plan || !plan->chunk || !bytes || cur0 < 0 || n_cur < 0 || (int64_t)cur0 + n_cur > plan->info.n_segments) return OCTO_EINVAL;
  const int64_t rows = plan->chunk->row0[cur0 + n_cur] - plan->chunk->row0[cur0];
  *bytes = octo::stat_bytes(rows) + octo::align_up((size_t)rows * 8, 256);
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
  if (n > 0 && (!ids || !ws || ws_bytes < need || ((uintptr_t)ws & 15))) return OCTO_EINVAL;
  if (n_cur == 0) return OCTO_OK;
  octo::VerifyParams p;
  p.x = logits, p.y = draft_logits;
  p.ld = ld, p.yld = draft_ld, p.eld = noise_ld;
  p.V = vocab;
  p.c = inv_temp, p.cy = draft_inv_temp;
  p.row0 = plan->seg_row_base + cur0;
  p.first = first;
  p.ids = ids, p.u = u, p.noise = noise;
  p.n_accept = n_accept, p.next_id = next_id, p.next_logp = next_logp, p.accept_p = accept_p;
  p.stat = static_cast<float2*>(ws);
  p.best = reinterpret_cast<unsigned long long*>(static_cast<char*>(ws) + octo::stat_bytes(n));
  p.n_rows = n;
  p.status = plan->pool->d_status;
  cudaStream_t s = (cudaStream_t)stream;
  plan->last_stream = s;
  if (dtype == OCTO_DTYPE_BF16)
    return greedy ? octo::run<__nv_bfloat16, true>(p, n_cur, s) : octo::run<__nv_bfloat16, false>(p, n_cur, s);
  return greedy ? octo::run<float, true>(p, n_cur, s) : octo::run<float, false>(p, n_cur, s);
}

}  // extern "C"
