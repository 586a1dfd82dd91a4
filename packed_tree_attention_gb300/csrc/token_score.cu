// Token scoring: the log-probabilities of given tokens, each row's entropy and its most
// likely alternatives, and the gradient of the first two.
//
// Row r of the logits x (V entries, c = inv_temp, m = max x):
//   S = sum_v exp(c (x_v - m)),  p_v = exp(c (x_v - m)) / S
//   logp[t] = c (x[id t] - m) - ln S  for the tokens t that r feeds (see SuccTable)
//   H = ln S - sum_v p_v c (x_v - m)
//   dx_v = c (sum over t with id t = v of g_t - p_v G - g_H p_v (ln p_v + H)),  G = sum_t g_t
// (m, ln S) is kept rather than m c + ln S: at logits in the thousands the sum's rounding
// would be a per-mille error of every probability that the gradient forms from it.

#include "row_common.cuh"

namespace octo {
namespace {

using namespace rows;

constexpr int kThreads = 512;

struct ScoreParams {
  const void* logits;
  int64_t ld;
  int32_t V, row0, k;
  float c;
  const int32_t* ids;    // [plan rows] or null
  float* logp;           // [plan rows] or null
  float* row_stat;       // [n][2]
  float* entropy;        // [n] or null
  int32_t* top_ids;      // [n][k]
  float* top_logp;       // [n][k]
  SuccTable succ;
  int32_t* status;
};

// One CTA per row: one pass for the statistics, then one pass per alternative for the
// largest entry after the last one found.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_token_score(ScoreParams p) {
  using VT = Vec<T>;
  __shared__ float red[96];
  __shared__ unsigned long long s_best;
  const int rl = blockIdx.x;
  const T* row = reinterpret_cast<const T*>(p.logits) + (size_t)rl * p.ld;
  const float c2 = p.c * kLog2e;
  Stat st;
  st.init();
  float mx = -INFINITY;
  for (int v = threadIdx.x; v < p.V; v += kThreads) {
    const float x = VT::get(row + v);
    mx = fmaxf(mx, x);
    if (x > st.m) st.rebase(x, c2);
    st.add(x, c2);
  }
  block_stat<kThreads>(st, c2, red);
  const bool empty = st.s == 0.f;
  const float m = empty ? -INFINITY : st.m, ls = empty ? -INFINITY : logf(st.s);
  auto term = [&](float x) { return x == -INFINITY ? -INFINITY : (x - m) * p.c - ls; };
  if (threadIdx.x == 0) {
    p.row_stat[2 * (size_t)rl] = m;
    p.row_stat[2 * (size_t)rl + 1] = ls;
    if (p.entropy) p.entropy[rl] = empty ? 0.f : ls - kLn2 * (st.a / st.s);
    if (p.ids) {
      int32_t t[kMaxSucc];
      bool start;
      const int n = p.succ.find(p.row0 + rl, t, &start);
      if (start) p.logp[p.row0 + rl] = 0.f;
      for (int i = 0; i < n; i++) {
        const int id = p.ids[t[i]];
        if (id < 0 || id >= p.V) {
          atomicExch(p.status, OCTO_EINVAL);
          p.logp[t[i]] = __int_as_float(0x7fc00000);
        } else {
          p.logp[t[i]] = term(VT::get(row + id));
        }
      }
    }
  }
  unsigned long long last = ~0ull;
  for (int j = 0; j < p.k; j++) {
    if (threadIdx.x == 0) s_best = 0;
    __syncthreads();
    unsigned long long best = 0;
    for (int v = threadIdx.x; v < p.V; v += kThreads) {
      const uint32_t key = order_key(VT::get(row + v));
      const unsigned long long e = ((unsigned long long)key << 32) | (uint32_t)~v;
      if (key && e < last && e > best) best = e;
    }
    atomicMax(&s_best, best);
    __syncthreads();
    last = s_best;
    if (threadIdx.x == 0) {
      const size_t o = (size_t)rl * p.k + j;
      p.top_ids[o] = last ? (int32_t) ~(uint32_t)last : -1;
      p.top_logp[o] = last ? term(order_value((uint32_t)(last >> 32))) : __int_as_float(0x7fc00000);
    }
    __syncthreads();
  }
}

struct ScoreBwdParams {
  const void* logits;
  void* dlogits;
  int64_t ld;
  int32_t V, row0;
  float c;
  const float* row_stat;
  const float* entropy;    // [n], with g_entropy
  const int32_t* ids;      // [plan rows], with g_logp
  const float* g_logp;     // [plan rows] or null
  const float* g_entropy;  // [n] or null
  SuccTable succ;
  int32_t* status;
};

// One CTA per row.  In log2 units, y = c2 (x - m) - log2 S and p = 2^y, an element's
// gradient is p (A + B y) with the row's A = -c (G + g_H H), B = -c g_H ln 2, plus
// c g_t at the successors' ids.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_token_score_bwd(ScoreBwdParams p) {
  using VT = Vec<T>;
  __shared__ int32_t s_id[kMaxSucc];
  __shared__ float s_g[kMaxSucc];
  __shared__ float s_G;
  __shared__ int32_t s_n;
  const int rl = blockIdx.x;
  const T* row = reinterpret_cast<const T*>(p.logits) + (size_t)rl * p.ld;
  T* grow = reinterpret_cast<T*>(p.dlogits) + (size_t)rl * p.ld;
  if (threadIdx.x == 0) {
    int n = 0;
    float G = 0.f;
    if (p.g_logp) {
      int32_t t[kMaxSucc];
      bool start;
      const int nt = p.succ.find(p.row0 + rl, t, &start);
      for (int i = 0; i < nt; i++) {
        const int id = p.ids[t[i]];
        if (id < 0 || id >= p.V) {
          atomicExch(p.status, OCTO_EINVAL);
          continue;
        }
        s_id[n] = id;
        s_g[n] = p.g_logp[t[i]];
        G += s_g[n++];
      }
    }
    s_n = n;
    s_G = G;
  }
  __syncthreads();
  const int n = s_n;
  const float m = p.row_stat[2 * (size_t)rl], ls = p.row_stat[2 * (size_t)rl + 1];
  const float gH = p.g_entropy ? p.g_entropy[rl] : 0.f, H = p.g_entropy ? p.entropy[rl] : 0.f;
  const bool empty = m == -INFINITY;
  const float c2 = p.c * kLog2e, l2 = ls * kLog2e;
  const float A = -p.c * (s_G + gH * H), B = -p.c * kLn2 * gH;
  for (int v = threadIdx.x; v < p.V; v += kThreads) {
    float g = 0.f;
    if (!empty) {
      const float y = max_nan((VT::get(row + v) - m) * c2 - l2, kCut);
      g = ex2f(y) * fmaf(B, y, A);
      for (int i = 0; i < n; i++)
        if (s_id[i] == v) g += p.c * s_g[i];
    }
    VT::put(grow + v, g);
  }
}

}  // namespace
}  // namespace octo

extern "C" {

int octo_token_score(octo_plan_t plan, int32_t row0, int32_t n_rows, const void* logits, int32_t dtype, int64_t ld,
                     int32_t vocab, float inv_temp, const int32_t* ids, float* logp, float* row_stat, float* entropy,
                     int32_t k, int32_t* top_ids, float* top_logp, void* stream) {
  using namespace octo;
  if (int st = check_rows(plan, row0, n_rows, logits, dtype, ld, vocab, inv_temp)) return st;
  if (!ids != !logp || k < 0 || k > kMaxTop || k > vocab || (k > 0 && (!top_ids || !top_logp))) return OCTO_EINVAL;
  if (ids && plan->max_succ > kMaxSucc) return OCTO_ENOTSUP;
  if (n_rows == 0) return OCTO_OK;
  if (!row_stat) return OCTO_EINVAL;
  ScoreParams p;
  p.logits = logits;
  p.ld = ld;
  p.V = vocab;
  p.row0 = row0;
  p.k = k;
  p.c = inv_temp;
  p.ids = ids;
  p.logp = logp;
  p.row_stat = row_stat;
  p.entropy = entropy;
  p.top_ids = top_ids;
  p.top_logp = top_logp;
  p.succ = succ_table(plan);
  p.status = plan->pool->d_status;
  cudaStream_t s = (cudaStream_t)stream;
  plan->last_stream = s;
  NvtxRange nv("octo_token_score");
  if (dtype == OCTO_DTYPE_BF16)
    k_token_score<__nv_bfloat16><<<n_rows, kThreads, 0, s>>>(p);
  else
    k_token_score<float><<<n_rows, kThreads, 0, s>>>(p);
  count_launch();
  return cuda_status(cudaGetLastError());
}

int octo_token_score_bwd(octo_plan_t plan, int32_t row0, int32_t n_rows, const void* logits, int32_t dtype, int64_t ld,
                         int32_t vocab, float inv_temp, const float* row_stat, const float* entropy, const int32_t* ids,
                         const float* g_logp, const float* g_entropy, void* dlogits, void* stream) {
  using namespace octo;
  if (int st = check_rows(plan, row0, n_rows, logits, dtype, ld, vocab, inv_temp)) return st;
  if ((g_logp && !ids) || (g_entropy && !entropy) || ((uintptr_t)dlogits & 15)) return OCTO_EINVAL;
  if (g_logp && plan->max_succ > kMaxSucc) return OCTO_ENOTSUP;
  if (n_rows == 0) return OCTO_OK;
  if (!row_stat || !dlogits) return OCTO_EINVAL;
  ScoreBwdParams p;
  p.logits = logits;
  p.dlogits = dlogits;
  p.ld = ld;
  p.V = vocab;
  p.row0 = row0;
  p.c = inv_temp;
  p.row_stat = row_stat;
  p.entropy = entropy;
  p.ids = ids;
  p.g_logp = g_logp;
  p.g_entropy = g_entropy;
  p.succ = succ_table(plan);
  p.status = plan->pool->d_status;
  cudaStream_t s = (cudaStream_t)stream;
  plan->last_stream = s;
  NvtxRange nv("octo_token_score_bwd");
  if (dtype == OCTO_DTYPE_BF16)
    k_token_score_bwd<__nv_bfloat16><<<n_rows, kThreads, 0, s>>>(p);
  else
    k_token_score_bwd<float><<<n_rows, kThreads, 0, s>>>(p);
  count_launch();
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
