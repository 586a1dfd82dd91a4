// Distillation from a teacher's top logits: the divergence of each row's student
// distribution from the teacher's listed entries, with its gradient.
//
// Row r: student q = softmax(c x) over V entries, c = inv_temp; teacher entries
// (id_i, z_i), i < k, with id_i < 0 or z_i = -inf an empty one.
//   renormalised: P_i = exp(c z_i) / sum_j exp(c z_j)
//   with the rest: P_i = exp(z_i), P_R = max(0, 1 - sum_i P_i)
//   KL = sum_i P_i (ln P_i - ln q_{id i}) + P_R (ln P_R - ln q_R),  q_R = sum of q outside
//        the listed ids
//   dKL/dx_v = c (q_v P - sum over i with id_i = v of P_i - [v not listed] P_R q_v / q_R),
//        P = sum_i P_i + P_R
// q_R is summed over the entries outside the list itself: 1 - sum_i q_i would lose it
// where the list holds nearly all of the mass.

#include "row_common.cuh"

namespace octo {
namespace {

using namespace rows;

constexpr int kThreads = 512;

struct DistillParams {
  const void* logits;
  void* dlogits;            // or null
  int64_t ld;
  int32_t V, row0, k, tail;
  float c, gs;
  const int32_t* t_ids;     // [n][k]
  const float* t_val;       // [n][k]
  const float* w;           // [plan rows] or null (ones)
  float* row_kl;            // [plan rows]
  float* part;              // [n] weighted row losses, or null
  int32_t* status;
};

// One CTA per row: a pass for the sums inside and outside the list, a pass for the gradient.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_distill(DistillParams p) {
  using VT = Vec<T>;
  __shared__ float red[96];
  __shared__ int32_t s_id[kMaxTop];
  __shared__ float s_p[kMaxTop];
  const int rl = blockIdx.x, tid = threadIdx.x;
  const T* row = reinterpret_cast<const T*>(p.logits) + (size_t)rl * p.ld;
  T* grow = p.dlogits ? reinterpret_cast<T*>(p.dlogits) + (size_t)rl * p.ld : nullptr;
  const float w = p.w ? p.w[p.row0 + rl] : 1.f;
  const float c2 = p.c * kLog2e;
  bool live = w != 0.f;
  // teacher entries
  float z = -INFINITY;
  int id = -1;
  if (tid < p.k) {
    id = p.t_ids[(size_t)rl * p.k + tid];
    z = p.t_val[(size_t)rl * p.k + tid];
    if (id >= p.V) atomicExch(p.status, OCTO_EINVAL);
    if (id < 0 || id >= p.V || z == -INFINITY) id = -1, z = -INFINITY;
    s_id[tid] = id;
  }
  float lp, P, pr = 0.f, zero = 0.f;
  if (p.tail) {
    lp = z;
    P = expf(z);
    float sum = P;
    block_sum2<kThreads>(sum, zero, red);
    pr = fmaxf(0.f, 1.f - sum);
    if (sum != sum) pr = sum;
  } else {
    Stat t{z == -INFINITY ? -FLT_MAX : z, z == -INFINITY ? 0.f : 1.f, 0.f};
    block_stat<kThreads>(t, c2, red);
    if (t.s == 0.f) live = false;
    lp = z == -INFINITY ? -INFINITY : (z - t.m) * p.c - logf(t.s);
    P = expf(lp);
  }
  if (tid < p.k) s_p[tid] = P;
  __syncthreads();
  float kl = 0.f, fix = 0.f;
  float mo = 0.f, lo = 0.f, fo = 0.f;   // reference and factor of the unlisted entries' gradient
  if (live) {
    // statistics of the entries that the list leaves out and of the listed ones (each id
    // once); without the rest term the two need not be told apart
    auto listed = [&](int v) {
      for (int i = 0; i < p.k; i++)
        if (s_id[i] == v) return true;
      return false;
    };
    Stat o, in;
    o.init();
    in.init();
    for (int v = tid; v < p.V; v += kThreads) {
      const float x = VT::get(row + v);
      Stat& st = p.tail && listed(v) ? in : o;
      if (x > st.m) st.rebase(x, c2);
      st.add(x, c2);
    }
    block_stat<kThreads>(o, c2, red);
    block_stat<kThreads>(in, c2, red);
    Stat all = o;
    all.merge(in.m, in.s, in.a, c2);
    if (all.s == 0.f) live = false;
    if (live) {
      const float ls = logf(all.s);
      float term = 0.f, sum = 0.f, lq = 0.f;
      if (id >= 0) {
        lq = (VT::get(row + id) - all.m) * p.c - ls;
        if (P != 0.f) term = P * (lp - lq), sum = P;
      }
      block_sum2<kThreads>(term, sum, red);
      kl = term;
      mo = o.m;
      if (o.s == 0.f) {
        pr = 0.f;   // nothing outside the list has mass
      } else {
        lo = logf(o.s);
        const float lqr = (o.m - all.m) * p.c + lo - ls;
        if (pr != 0.f) kl += pr * (logf(pr) - lqr);
        fo = expf(lqr) * (sum + pr) - pr;
      }
      fix = expf(lq) * (sum + pr);
    }
  }
  const float f = p.gs * w * p.c;
  if (tid == 0) {
    p.row_kl[p.row0 + rl] = kl;
    if (p.part) p.part[rl] = live ? w * kl : 0.f;
  }
  if (!grow) return;
  __syncthreads();  // the listed entries are read before the gradient may overwrite them
  const float l2 = lo * kLog2e;
  for (int v = tid; v < p.V; v += kThreads)
    VT::put(grow + v, live ? f * fo * ex2f(max_nan((VT::get(row + v) - mo) * c2 - l2, kCut)) : 0.f);
  __syncthreads();
  // the listed entries, each id by its first entry
  if (live && id >= 0) {
    float sub = 0.f;
    bool first = true;
    for (int i = 0; i < p.k; i++)
      if (s_id[i] == id) sub += s_p[i], first = first && i >= tid;
    if (first) VT::put(grow + id, f * (fix - sub));
  }
}

}  // namespace
}  // namespace octo

extern "C" {

int octo_distill_topk_workspace_size(int32_t n_rows, size_t* bytes) {
  if (n_rows < 0 || !bytes) return OCTO_EINVAL;
  *bytes = octo::align_up((size_t)n_rows * sizeof(float), 256);
  return OCTO_OK;
}

int octo_distill_topk(octo_plan_t plan, int32_t row0, int32_t n_rows, const void* logits, int32_t dtype, int64_t ld,
                      int32_t vocab, float inv_temp, int32_t k, const int32_t* teach_ids, const float* teach_val,
                      int32_t tail, const float* weight, float* row_kl, void* dlogits, float grad_scale, float* loss,
                      void* ws, size_t ws_bytes, void* stream) {
  using namespace octo;
  if (int st = check_rows(plan, row0, n_rows, logits, dtype, ld, vocab, inv_temp)) return st;
  if (k < 1 || k > kMaxTop || ((uintptr_t)dlogits & 15)) return OCTO_EINVAL;
  cudaStream_t s = (cudaStream_t)stream;
  if (n_rows == 0) {
    if (loss) OCTO_CUDA(cudaMemsetAsync(loss, 0, sizeof(float), s));
    return OCTO_OK;
  }
  size_t need = 0;
  octo_distill_topk_workspace_size(n_rows, &need);
  if (!teach_ids || !teach_val || !row_kl || (loss && (!ws || ws_bytes < need))) return OCTO_EINVAL;
  DistillParams p;
  p.logits = logits;
  p.dlogits = dlogits;
  p.ld = ld;
  p.V = vocab;
  p.row0 = row0;
  p.k = k;
  p.tail = tail ? 1 : 0;
  p.c = inv_temp;
  p.gs = grad_scale;
  p.t_ids = teach_ids;
  p.t_val = teach_val;
  p.w = weight;
  p.row_kl = row_kl;
  p.part = loss ? (float*)ws : nullptr;
  p.status = plan->pool->d_status;
  plan->last_stream = s;
  NvtxRange nv("octo_distill_topk");
  if (dtype == OCTO_DTYPE_BF16)
    k_distill<__nv_bfloat16><<<n_rows, kThreads, 0, s>>>(p);
  else
    k_distill<float><<<n_rows, kThreads, 0, s>>>(p);
  count_launch();
  if (int st = cuda_status(cudaGetLastError())) return st;
  return loss ? launch_loss_sum((const float*)ws, n_rows, loss, s) : OCTO_OK;
}

}  // extern "C"
