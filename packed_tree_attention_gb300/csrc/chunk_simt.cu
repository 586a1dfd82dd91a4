// Chunk attention on the CUDA cores (fp32 pools, page sizes without 64-key blocks), and the
// joining of partial results for both kernel families.
//
// softmax(scale q K^T) V of the rows of one tile and kv head, one pass over the tile's blocks
// with the running maximum m and sum l of each row (log2 domain): with m' = max(m, block's max),
//     l <- l 2^(m - m') + sum 2^(s - m'),   O <- O 2^(m - m') + P V.
// A CTA has 16 RM rows (token * G + head), staged with 64 keys at a time in shared memory as
// fp32.  Thread (ty, tx) of 16 x 16 holds rows ty + 16 i and keys tx + 16 j of the scores (RM x
// 4 of them, each as a pair of sums over even and odd places), then columns 4 tx + 64 c .. + 3 of
// O, two fp32 operations an instruction: 4 RM and RM D / 16 accumulators against RM + 4 and RM / 4
// + D / 64 vector loads for each four steps of the inner product.  fp32 pools are copied with
// cp.async, the next K while P V runs and the next V while S does.  Everything is fp32.
// Bound by latency: at d 128 an SM holds one CTA from RM = 4 on, two warps a scheduler, which wait for
// shared memory and for the instruction before.  200 new tokens of two cursors behind 4,096, 16 query
// heads: 493 us, 28 TFLOP/s; the FMA pipe is busy 47% of the time, shared memory 60%, an
// instruction is issued in 40% of the cycles, barriers are 3% of the warps' waiting.  Single tokens
// behind 14,000: 154 us, 1.2 TB/s.

#include <cuda_bf16.h>

#include <algorithm>

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
  int32_t Hq, Hkv, G, P, span, window, n_sub;   // span: keys of a block in one page
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

__device__ __forceinline__ void copy16(float* dst, const float* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

template <typename T, int D, int RM>
__global__ void __launch_bounds__(256) k_chunk_simt(const __grid_constant__ SimtParams p) {
  using rows::f2;
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
  f2 o[RM][C][2];
#pragma unroll
  for (int i = 0; i < RM; i++) {
    own[i] = t.t0 + min(r0 + ty + 16 * i, R - 1) / p.G;
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < C; c++) o[i][c][0] = o[i][c][1] = 0;
  }
  const int first = t.t0 + r0 / p.G, last = t.t0 + (min(r0 + M, R) - 1) / p.G;
  // the steps: 64 slots of a block at a time, where some row of the CTA sees one
  struct Step {
    int b, j0, lo, hi;              // slots that some row sees
    int own0, seen, k_lo, k_hi;     // of the block
  };
  auto lowest = [&](const Step& s, int i) {   // slots [lowest, highest) that the row at own index i sees
    return p.window > 0 ? max(s.k_lo, i + t.shift - p.window + 1 - s.seen) : s.seen <= i ? s.k_lo : s.k_hi;
  };
  auto highest = [&](const Step& s, int i) { return min(s.k_hi, i - s.own0 + 1); };
  auto enter = [&](Step& s) {   // at block s.b or the next one with such a slot
    for (; s.b < t.n; s.b++) {
      const int4 k = *reinterpret_cast<const int4*>(&p.blocks[t.blk + s.b].own0);
      s.own0 = k.x, s.seen = k.y, s.k_lo = k.z & 0xffff, s.k_hi = (uint32_t)k.z >> 16;
      s.lo = lowest(s, p.window > 0 ? first : last), s.hi = highest(s, last);
      s.j0 = s.lo / kKeys * kKeys;
      if (s.j0 < s.hi) return;
    }
  };
  auto advance = [&](Step& s) {
    s.j0 += kKeys;
    if (s.j0 >= s.hi) s.b++, enter(s);
  };
  auto load = [&](const Step& s, const void* pool, float* dst, int ld) {
    const ChunkBlock* k = p.blocks + t.blk + s.b;
    const int slot0 = k->slot0;
    for (int i = tid; i < kKeys * (D / 4); i += 256) {
      const int j = i / (D / 4), c = i % (D / 4) * 4, slot = s.j0 + j;
      const bool live = slot >= s.lo && slot < s.hi;
      const int at = live ? slot : s.lo;
      const T* src = static_cast<const T*>(pool) + (((size_t)k->page[at / p.span] * p.Hkv + g) * p.P + slot0 + at % p.span) * D + c;
      if constexpr (sizeof(T) == 4) copy16(dst + j * ld + c, reinterpret_cast<const float*>(src), live);
      else *reinterpret_cast<float4*>(dst + j * ld + c) = live ? load4(src) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    copies_issued();
  };
  Step s;
  s.b = 0;
  enter(s);
  if (s.b < t.n) {
    load(s, p.k, sk, LD);
    load(s, p.v, sv, D);
  }
  while (s.b < t.n) {
    Step next = s;
    advance(next);
    copies_wait<1>();   // K of this step
    __syncthreads();
    f2 a2[RM][4];
#pragma unroll
    for (int i = 0; i < RM; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) a2[i][j] = 0;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      ulonglong2 y[4];
#pragma unroll
      for (int j = 0; j < 4; j++) y[j] = *reinterpret_cast<const ulonglong2*>(sk + (tx + 16 * j) * LD + c);
#pragma unroll
      for (int i = 0; i < RM; i++) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(sq + (ty + 16 * i) * LD + c);
#pragma unroll
        for (int j = 0; j < 4; j++) a2[i][j] = rows::fma2(x.y, y[j].y, rows::fma2(x.x, y[j].x, a2[i][j]));
      }
    }
    __syncthreads();    // K is read
    if (next.b < t.n) load(next, p.k, sk, LD);
    else copies_issued();
#pragma unroll
    for (int i = 0; i < RM; i++) {
      const int lo = lowest(s, own[i]), hi = highest(s, own[i]);
      float mx = m[i], x[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int slot = s.j0 + tx + 16 * j;
        float e, f;
        rows::unpack2(a2[i][j], e, f);
        x[j] = slot >= lo && slot < hi ? (e + f) * p.scale_log2 : -INFINITY;
        mx = fmaxf(mx, x[j]);
      }
#pragma unroll
      for (int w = 8; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float base = mx == -INFINITY ? 0.f : mx;
      const float f = ex2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const float e2 = ex2f(x[j] - base);
        sum += e2;
        sp[(ty + 16 * i) * LP + tx + 16 * j] = e2;
      }
      l[i] = l[i] * f + sum;   // the lane's own part of the row's sum
      m[i] = mx;
      const f2 ff = rows::pack2(f, f);
#pragma unroll
      for (int c = 0; c < C; c++) o[i][c][0] = rows::mul2(o[i][c][0], ff), o[i][c][1] = rows::mul2(o[i][c][1], ff);
    }
    copies_wait<1>();   // V of this step
    __syncthreads();
#pragma unroll 2
    for (int j = 0; j < kKeys; j += 4) {
      float4 w[RM];
#pragma unroll
      for (int i = 0; i < RM; i++) w[i] = *reinterpret_cast<const float4*>(sp + (ty + 16 * i) * LP + j);
#pragma unroll
      for (int jj = 0; jj < 4; jj++) {
        ulonglong2 y[C];
#pragma unroll
        for (int c = 0; c < C; c++) y[c] = *reinterpret_cast<const ulonglong2*>(sv + (j + jj) * D + 64 * c + 4 * tx);
#pragma unroll
        for (int i = 0; i < RM; i++) {
          const float e2 = jj == 0 ? w[i].x : jj == 1 ? w[i].y : jj == 2 ? w[i].z : w[i].w;
          const f2 ee = rows::pack2(e2, e2);
#pragma unroll
          for (int c = 0; c < C; c++) {
            o[i][c][0] = rows::fma2(ee, y[c].x, o[i][c][0]);
            o[i][c][1] = rows::fma2(ee, y[c].y, o[i][c][1]);
          }
        }
      }
    }
    __syncthreads();    // P and V are read
    if (next.b < t.n) load(next, p.v, sv, D);
    else copies_issued();
    s = next;
  }
  copies_wait<0>();
#pragma unroll
  for (int i = 0; i < RM; i++) {
    const int r = r0 + ty + 16 * i;
    float sum = l[i];
#pragma unroll
    for (int w = 8; w; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    if (r >= R) continue;
    auto columns = [&](int c) {
      float4 v;
      rows::unpack2(o[i][c][0], v.x, v.y);
      rows::unpack2(o[i][c][1], v.z, v.w);
      return v;
    };
    if (t.part >= 0) {
      const int64_t at = (int64_t)t.part + r;
#pragma unroll
      for (int c = 0; c < C; c++) *reinterpret_cast<float4*>(p.part + at * D + 64 * c + 4 * tx) = columns(c);
      if (tx == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(m[i], sum);
    } else {
      const size_t at = (size_t)(t.row0 + r / p.G) * p.Hq + g * p.G + r % p.G;
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int c = 0; c < C; c++) {
        const float4 v = columns(c);
        store4(static_cast<T*>(p.out) + at * D + 64 * c + 4 * tx, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
      }
      if (tx == 0 && p.lse) p.lse[at] = sum == 0.f ? -INFINITY : (m[i] + log2f(sum)) * 0.69314718055994531f;   // NaN: NaN
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
  if (lane == 0 && lse) lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;   // NaN: NaN
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
  // rows of a CTA, 16 rm: a step takes about rm + 1.5 units, and the SMs take the CTAs in turn
  const int R = plan->chunk->max_rows * p.G, sms = std::max(1, rows::sm_count());
  int rm = 1;
  double best = 0;
  for (int x : {1, 2, 3, 4, 5, 6, 8}) {
    const int64_t ctas = plan->chunk->simt_ctas[x];
    const double t = std::max((double)((ctas + sms - 1) / sms), ctas > 2 * sms ? (double)ctas / sms + 0.5 : 0.0) * (x + 1.5);
    if (x == 1 || t <= best) rm = x, best = t;
  }
  p.n_sub = (R + 16 * rm - 1) / (16 * rm);
  const int64_t ctas = (int64_t)plan->chunk->n_work * p.n_sub;
  if (ctas > INT32_MAX) return OCTO_EINVAL;
  switch (rm) {
    case 1: return launch<T, D, 1>(p, ctas, s);
    case 2: return launch<T, D, 2>(p, ctas, s);
    case 3: return launch<T, D, 3>(p, ctas, s);
    case 4: return launch<T, D, 4>(p, ctas, s);
    case 5: return launch<T, D, 5>(p, ctas, s);
    case 6: return launch<T, D, 6>(p, ctas, s);
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
  p.Hq = c.Hq, p.Hkv = d.n_kv_heads, p.G = c.G, p.P = d.page_size;
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
