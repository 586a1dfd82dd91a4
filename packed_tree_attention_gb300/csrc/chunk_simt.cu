// Chunk attention on the CUDA cores (fp32 pools, page sizes without 64-key blocks), and the
// joining of partial results for both kernel families.
//
// softmax(scale q K^T) V of the rows of one tile and kv head, one pass over the tile's blocks
// with the running maximum m and sum l of each row (log2 domain): with m' = max(m, block's max),
//     l <- l 2^(m - m') + sum 2^(s - m'),   O <- O 2^(m - m') + P V.
// A CTA has 16 RM rows (token * G + head), staged with 64 keys at a time in shared memory as
// fp32.  Thread (ty, tx) of 16 x 16 holds rows ty + 16 i and keys tx + 16 j of the scores (RM x
// 4 of them), then columns 4 tx + 64 c .. + 3 of O: 4 RM and RM D / 16 accumulators against RM +
// 4 and RM / 4 + D / 64 vector loads for each four steps of the inner product, so that from RM =
// 4 on the FMAs and not shared memory bound it.  Everything is fp32.

#include <cuda_bf16.h>

#include "chunk.h"
#include "row_ring.cuh"

namespace octo {
namespace {

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct SimtParams {
  const ChunkBlock* blocks;
  const ChunkWork* work;
  const void *q, *k, *v;
  void* out;
  float *lse, *part, *part_ml;
  int32_t Hq, Hkv, G, P, span, width, window, n_sub;   // span: keys of a block in one page
  float scale_log2;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}

constexpr int kKeys = 64;                       // keys staged at a time
template <int D, int RM>
constexpr int simt_smem() {
  return (16 * RM * (D + 4) + kKeys * (D + 4) + kKeys * D + 16 * RM * (kKeys + 4)) * (int)sizeof(float);
}

template <typename T, int D, int RM>
__global__ void __launch_bounds__(256) k_chunk_simt(const __grid_constant__ SimtParams p) {
  constexpr int M = 16 * RM, C = D / 64, LD = D + 4, LP = kKeys + 4;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;
  float* sk = sq + M * LD;
  float* sv = sk + kKeys * LD;
  float* sp = sv + kKeys * D;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int sub = blockIdx.x % p.n_sub;
  const ChunkWork t = p.work[blockIdx.x / p.n_sub];
  const int g = t.g;
  const int R = t.rows * p.G, r0 = sub * M;
  if (r0 >= R) return;
  const T* q = static_cast<const T*>(p.q);
  for (int i = tid; i < M * (D / 4); i += 256) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < R) {
      const int tok = (r0 + r) / p.G, h = (r0 + r) % p.G;
      x = load4(q + ((size_t)(t.row0 + tok) * p.Hq + g * p.G + h) * D + c);
    }
    *reinterpret_cast<float4*>(sq + r * LD + c) = x;
  }
  int own[RM];          // own index of the thread's rows
  float m[RM], l[RM];
  float4 o[RM][C];
#pragma unroll
  for (int i = 0; i < RM; i++) {
    own[i] = t.t0 + min(r0 + ty + 16 * i, R - 1) / p.G;
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < C; c++) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int first = t.t0 + r0 / p.G, last = t.t0 + (min(r0 + M, R) - 1) / p.G;
  for (int b = 0; b < t.n; b++) {
    const ChunkBlock k = p.blocks[t.blk + b];
    int lo, hi, unused;   // what some row of the CTA sees
    chunk_range(k, first, first + t.shift - p.window + 1, p.window > 0, lo, unused);
    chunk_range(k, last, 0, false, unused, hi);
    for (int j0 = lo / kKeys * kKeys; j0 < hi; j0 += kKeys) {
      __syncthreads();
      for (int i = tid; i < kKeys * (D / 4); i += 256) {
        const int j = i / (D / 4), c = i % (D / 4) * 4, slot = j0 + j;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (slot >= lo && slot < hi) {
          const size_t row = ((size_t)k.page[slot / p.span] * p.Hkv + g) * p.P + k.slot0 + slot % p.span;
          x = load4(static_cast<const T*>(p.k) + row * D + c);
          y = load4(static_cast<const T*>(p.v) + row * D + c);
        }
        *reinterpret_cast<float4*>(sk + j * LD + c) = x;
        *reinterpret_cast<float4*>(sv + j * D + c) = y;
      }
      __syncthreads();
      float s[RM][4];
#pragma unroll
      for (int i = 0; i < RM; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) s[i][j] = 0.f;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 x[RM], y[4];
#pragma unroll
        for (int i = 0; i < RM; i++) x[i] = *reinterpret_cast<const float4*>(sq + (ty + 16 * i) * LD + c);
#pragma unroll
        for (int j = 0; j < 4; j++) y[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * LD + c);
#pragma unroll
        for (int i = 0; i < RM; i++)
#pragma unroll
          for (int j = 0; j < 4; j++)
            s[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, s[i][j]))));
      }
#pragma unroll
      for (int i = 0; i < RM; i++) {
        int a, e;
        chunk_range(k, own[i], own[i] + t.shift - p.window + 1, p.window > 0, a, e);
        float mx = m[i];
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const int slot = j0 + tx + 16 * j;
          s[i][j] = slot >= a && slot < e ? s[i][j] * p.scale_log2 : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int w = 8; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float base = mx == -INFINITY ? 0.f : mx;
        const float f = ex2f(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float e2 = ex2f(s[i][j] - base);
          sum += e2;
          sp[(ty + 16 * i) * LP + tx + 16 * j] = e2;
        }
        l[i] = l[i] * f + sum;   // the lane's own part of the row's sum
        m[i] = mx;
#pragma unroll
        for (int c = 0; c < C; c++) o[i][c].x *= f, o[i][c].y *= f, o[i][c].z *= f, o[i][c].w *= f;
      }
      __syncwarp();   // a row's 16 lanes are in one warp
#pragma unroll 2
      for (int j = 0; j < kKeys; j += 4) {
        float4 w[RM];
#pragma unroll
        for (int i = 0; i < RM; i++) w[i] = *reinterpret_cast<const float4*>(sp + (ty + 16 * i) * LP + j);
#pragma unroll
        for (int jj = 0; jj < 4; jj++)
#pragma unroll
          for (int c = 0; c < C; c++) {
            const float4 y = *reinterpret_cast<const float4*>(sv + (j + jj) * D + 64 * c + 4 * tx);
#pragma unroll
            for (int i = 0; i < RM; i++) {
              const float e2 = jj == 0 ? w[i].x : jj == 1 ? w[i].y : jj == 2 ? w[i].z : w[i].w;
              o[i][c].x = fmaf(e2, y.x, o[i][c].x);
              o[i][c].y = fmaf(e2, y.y, o[i][c].y);
              o[i][c].z = fmaf(e2, y.z, o[i][c].z);
              o[i][c].w = fmaf(e2, y.w, o[i][c].w);
            }
          }
      }
      __syncwarp();   // P is read before the next scores' replaces it
    }
  }
#pragma unroll
  for (int i = 0; i < RM; i++) {
    const int r = r0 + ty + 16 * i;
    float sum = l[i];
#pragma unroll
    for (int w = 8; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    if (r >= R) continue;
    if (t.part >= 0) {
      const int64_t at = (int64_t)t.part + r;
#pragma unroll
      for (int c = 0; c < C; c++) *reinterpret_cast<float4*>(p.part + at * D + 64 * c + 4 * tx) = o[i][c];
      if (tx == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(m[i], sum);
    } else {
      const size_t at = (size_t)(t.row0 + r / p.G) * p.Hq + g * p.G + r % p.G;
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int c = 0; c < C; c++)
        store4(static_cast<T*>(p.out) + at * D + 64 * c + 4 * tx,
               make_float4(o[i][c].x * inv, o[i][c].y * inv, o[i][c].z * inv, o[i][c].w * inv));
      if (tx == 0 && p.lse) p.lse[at] = sum > 0.f ? (m[i] + log2f(sum)) * 0.69314718055994531f : -INFINITY;
    }
  }
}

// Joined rows: the partial sums and outputs relative to the common maximum, in the refs' order.
// `team` warps of a CTA's eight take a row: each the partial results i = w mod team, whose sums
// the first of them adds up.  Bound by the latency of the partial results' loads.
template <typename T, int D>
__global__ void __launch_bounds__(256) k_chunk_join(const ChunkJoin* joins, const int32_t* refs, const float* part,
                                                   const float* part_ml, T* out, float* lse, int Hq, int G, int team) {
  constexpr int E = D / 32;
  __shared__ float s_o[8][D];
  __shared__ float s_l[8];
  const ChunkJoin jn = joins[blockIdx.x];
  const int g = jn.g, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % team;
  const int R = jn.rows * G, r = blockIdx.y * (8 / team) + warp / team;
  const bool live = r < R;
  rows::launch_dependents();
  rows::wait_for_predecessor();
  auto place = [&](int i) { return (int64_t)refs[jn.ref0 + i] + r; };
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; e++) o[e] = 0.f;
  if (live) {
    for (int i = lane; i < jn.n_refs; i += 32) m = fmaxf(m, part_ml[2 * place(i)]);
#pragma unroll
    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 4
    for (int i = w; i < jn.n_refs; i += team) {
      const int64_t at = place(i);
      const float2 ml = *reinterpret_cast<const float2*>(part_ml + 2 * at);
      const float f = ex2f(ml.x - base);
      l = fmaf(ml.y, f, l);
      const float* src = part + at * D + lane * E;
      float x[E];
      if (E == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        x[0] = v.x, x[1] = v.y, x[E - 2] = v.z, x[E - 1] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        x[0] = v.x, x[1] = v.y;
      }
#pragma unroll
      for (int e = 0; e < E; e++) o[e] = fmaf(x[e], f, o[e]);
    }
  }
  if (team > 1) {
    if (w) {
#pragma unroll
      for (int e = 0; e < E; e++) s_o[warp][lane * E + e] = o[e];
      if (lane == 0) s_l[warp] = l;
    }
    __syncthreads();
    if (w) return;
    for (int k = 1; k < team; k++) {
      l += s_l[warp + k];
#pragma unroll
      for (int e = 0; e < E; e++) o[e] += s_o[warp + k][lane * E + e];
    }
  }
  if (!live) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const size_t row = (size_t)(jn.row0 + r / G) * Hq + g * G + r % G;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    T* dst = out + row * D + lane * E + e;
    if (sizeof(T) == 2)
      *reinterpret_cast<__nv_bfloat162*>(dst) = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
    else
      *reinterpret_cast<float2*>(dst) = make_float2(o[e] * inv, o[e + 1] * inv);
  }
  if (lane == 0 && lse) lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

template <typename T, int D, int RM>
int launch(const SimtParams& p, int64_t ctas, cudaStream_t s) {
  constexpr int smem = simt_smem<D, RM>();
  if (int st = set_smem_limit((const void*)k_chunk_simt<T, D, RM>, smem)) return st;
  k_chunk_simt<T, D, RM><<<(unsigned)ctas, 256, smem, s>>>(p);
  count_launch();
  return cuda_status(cudaGetLastError());
}

template <typename T, int D>
int run(SimtParams p, const octo_plan_s* plan, cudaStream_t s) {
  // rows of a CTA: as many as the longest tile has, 128 at most
  const int R = plan->chunk->max_rows * p.G;
  const int rm = R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8;
  p.n_sub = (R + 16 * rm - 1) / (16 * rm);
  const int64_t ctas = (int64_t)plan->chunk->n_work * p.n_sub;
  if (ctas > INT32_MAX) return OCTO_EINVAL;
  switch (rm) {
    case 1: return launch<T, D, 1>(p, ctas, s);
    case 2: return launch<T, D, 2>(p, ctas, s);
    case 4: return launch<T, D, 4>(p, ctas, s);
    default: return launch<T, D, 8>(p, ctas, s);
  }
}

}  // namespace

int chunk_simt(const octo_plan_s* plan, const ChunkArgs& a, cudaStream_t s) {
  const octo_pool_desc& d = plan->pool->desc;
  const ChunkPlan& c = *plan->chunk;
  SimtParams p;
  p.blocks = c.blocks, p.work = c.work;
  p.q = a.q, p.k = a.k, p.v = a.v, p.out = a.out, p.lse = a.lse, p.part = a.part, p.part_ml = a.part_ml;
  p.Hq = c.Hq, p.Hkv = d.n_kv_heads, p.G = c.G, p.P = d.page_size, p.width = c.width;
  p.span = d.page_size < c.width ? d.page_size : c.width;
  p.window = c.window;
  p.n_sub = 1;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  if (d.dtype == OCTO_DTYPE_F32)
    return d.head_dim == 64 ? run<float, 64>(p, plan, s) : run<float, 128>(p, plan, s);
  return d.head_dim == 64 ? run<__nv_bfloat16, 64>(p, plan, s) : run<__nv_bfloat16, 128>(p, plan, s);
}

int chunk_join(const octo_plan_s* plan, const ChunkArgs& a, cudaStream_t s) {
  const octo_pool_desc& d = plan->pool->desc;
  const ChunkPlan& c = *plan->chunk;
  // up to four partial results are one round of loads for a warp
  const int team = c.max_refs <= 4 ? 1 : c.max_refs <= 8 ? 2 : c.max_refs <= 16 ? 4 : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)c.n_joins, (unsigned)((c.max_join_rows * c.G * team + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel, auto* out) {
    return cudaLaunchKernelEx(&cfg, kernel, (const ChunkJoin*)c.joins, (const int32_t*)c.refs, (const float*)a.part,
                              (const float*)a.part_ml, out, a.lse, (int)c.Hq, (int)c.G, team);
  };
  cudaError_t e;
  if (d.dtype == OCTO_DTYPE_F32)
    e = d.head_dim == 64 ? go(k_chunk_join<float, 64>, static_cast<float*>(a.out)) : go(k_chunk_join<float, 128>, static_cast<float*>(a.out));
  else
    e = d.head_dim == 64 ? go(k_chunk_join<__nv_bfloat16, 64>, static_cast<__nv_bfloat16*>(a.out))
                         : go(k_chunk_join<__nv_bfloat16, 128>, static_cast<__nv_bfloat16*>(a.out));
  count_launch();
  return cuda_status(e);
}

}  // namespace octo
