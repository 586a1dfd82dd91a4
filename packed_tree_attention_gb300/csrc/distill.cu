// Distillation from a teacher's top logits: the divergence of each row's student
// distribution from the teacher's listed entries, with its gradient.
//
// Row r: student q = softmax(c x) over V entries, c = inv_temp; teacher entries
// (id_i, z_i), i < k, with id_i < 0 or z_i = -inf an empty one.
//   renormalised: P_i = exp(c z_i) / sum_j exp(c z_j)
//   with the rest: P_i = exp(z_i), P_R = max(0, 1 - sum_i P_i)
//   T_v = sum over i with id_i = v of P_i
//   KL = sum over listed v of T_v (ln T_v - ln q_v) + P_R (ln P_R - ln q_R),  q_R = sum of q
//        outside the listed ids
//   dKL/dx_v = c (q_v P - T_v - [v not listed] P_R q_v / q_R),  P = sum_i P_i + P_R
// q_R is summed over the entries outside the list itself: 1 - sum_i q_i would lose it
// where the list holds nearly all of the mass.  For that, the consumers leave out every
// 16-byte vector that holds a listed id (a bit each in a table of the row's vectors), and a
// finisher adds what those hold besides.  The gradient pass writes every entry as an unlisted
// one, and the finisher then writes the listed ones.
// With the rest class the divergence is summed as sum of (P d - P + q), d = ln P - ln q, whose
// terms are never negative (share below): 240 rows of 30,000 fp32 entries with divergences
// around 2e-5 come out 3e-5 of them off, and 2e-3 by the plain sum.
//
// Bound by memory: V entries read and, for the gradient, V written; the second reading comes
// from L2.  Measured (16,384-byte stages, one GB300, 6.78 TB/s copied): 8,192 rows of 151,936
// bf16 against 64 entries 768 us with the gradient (6.5 TB/s of those bytes; 816 us with the rest
// class), 1,024 rows and 32 entries without it 56 us (5.6 TB/s), 500 rows of 50,001 fp32 with the
// rest class 40 us (5.0 TB/s).  Parts held in shared memory between the passes, which spares L2 the second
// reading, took 876 us: they leave too little of the ring for the copies to run ahead.

#include "row_ring.cuh"

namespace octo {
namespace {

using namespace rows;

struct DistillParams {
  const void* logits;
  void* dlogits;            // or null
  int64_t ld;
  int32_t V, row0, n, k, tail;
  float c, gs;
  const int32_t* t_ids;     // [n][k]
  const float* t_val;       // [n][k]
  const float* w;           // [plan rows] or null (ones)
  float* row_kl;            // [plan rows]
  float* part;              // [n] weighted row losses, or null
  int32_t* status;
  RingShape ring;
  int32_t words;            // words of the bitmap of a part's vectors
};

// What the gradient pass needs of a row: an entry outside the list has the gradient
// f 2^(c2 x - hi), or f 2^(c2 (x - m) - l2) where c2 m leaves the usual range.
struct RowScale {
  float f, hi, m, l2;
  int32_t live, usual;
};
// ln of the least probability that 64 bits hold.  Where every id outside the list is below it
// (masked with -inf, the type's lowest value or another far one), the rest class is dropped.
constexpr float kNoMass = -745.13f;
constexpr int kHashWords = 64;   // of the test for entries in one vector

// Of each finisher warp: the entries of its row, and the CTAs' sums, of every other of its rows.
struct __align__(16) WarpSmem {
  uint32_t hash[kHashWords];
  float x[kMaxTop];
  float in[2][kMaxCluster][4];
};
struct DistillSmem {
  RingBars bars;
  float part[kMaxRows][kConsWarps][2];
  RowScale scale[kMaxRows];
  WarpSmem warp[kFinishers];
};
constexpr int kBitmapOffset = ((int)sizeof(DistillSmem) + 127) / 128 * 128;
__host__ __device__ constexpr int slots_offset(int words) { return kBitmapOffset + (kMaxRows * words * 4 + 127) / 128 * 128; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(v) : "f"(v));
  return v;
}

// ln s = hi + lo, hi exact: a divergence is the small difference of large logarithms, and s
// rounded to one float would be felt in it.
__device__ __forceinline__ void split_log(float s, float* hi, float* lo) {
  const int e = (__float_as_int(s) >> 23) - 127;
  const float f = __int_as_float((__float_as_int(s) & 0x7fffff) | 0x3f800000);
  const bool normal = s >= FLT_MIN && s <= FLT_MAX;
  // ln 2 = 355 / 512 + a rest (Cody and Waite's reduction): e * 355 / 512 is exact
  *hi = normal ? (float)e * (355.f / 512.f) : logf(s);
  *lo = normal ? fmaf((float)e, (float)(0.69314718055994531 - 355.0 / 512.0), logf(f)) : 0.f;
}

// A class's share of a divergence whose classes hold all of both masses: P d + (q - P), d = ln P - ln q.
// The terms added are 0 in sum, and each share is P (d + e^-d - 1) >= 0, of second order in d:
// an error of d is felt times d only.  Near a student that has learnt its teacher the plain sum
// of P d is the small rest of terms of both signs.
__device__ __forceinline__ float share(float P, float d, float q) {
  if (!(fabsf(d) < 0.5f)) return P == 0.f ? q : P * d + (q - P);
  // the power series from d^2 / 2 on; what is left out is below 3e-9 of it
  float h = -1.f / 362880;
  h = fmaf(h, d, 1.f / 40320);
  h = fmaf(h, d, -1.f / 5040);
  h = fmaf(h, d, 1.f / 720);
  h = fmaf(h, d, -1.f / 120);
  h = fmaf(h, d, 1.f / 24);
  h = fmaf(h, d, -1.f / 6);
  h = fmaf(h, d, 0.5f);
  return P * d * d * h;
}

// With a gradient every row is streamed twice, the first pass of the next row before the second
// of this one, so that the join of a row's sums is not waited for.  The second time a row comes
// from L2.
// kEntries: entries of a lane, at least k / 32.
template <typename T, bool kGrad, int kEntries>
__global__ void __launch_bounds__(kBlock, 1) k_distill(const __grid_constant__ DistillParams p) {
  using VT = Vec<T>;
  constexpr int E = VT::E;
  extern __shared__ __align__(128) uint8_t smem[];
  DistillSmem& ss = *reinterpret_cast<DistillSmem*>(smem);
  uint32_t* const bitmap = reinterpret_cast<uint32_t*>(smem + kBitmapOffset);
  uint4* const slots = reinterpret_cast<uint4*>(smem + slots_offset(p.words));
  RingBars& bar = ss.bars;
  const RingShape rs = p.ring;
  const uint32_t rank = rs.cs > 1 ? cluster_rank() : 0;
  const int n_clusters = gridDim.x / rs.cs, cluster = blockIdx.x / rs.cs;
  const int nv = p.V / E;
  const int v0 = min(nv, (int)rank * rs.seg), nvec = min(rs.seg, nv - v0);
  const int tid = threadIdx.x, lane = tid & 31;
  const float c2 = p.c * kLog2e;
  const T* const logits = reinterpret_cast<const T*>(p.logits);
  T* const dlogits = reinterpret_cast<T*>(p.dlogits);
  auto weight = [&](int r) { return !p.w ? 1.f : r < p.n ? p.w[p.row0 + r] : 0.f; };

  if (tid == 0) bar.init(1);
  __syncthreads();
  if (rs.cs > 1) cluster_sync();
  wait_for_predecessor();

  if (tid >= kCopy && tid < kFirstCons) {
    // ---- copies (rows of weight 0 are not read) ----
    if (tid == kCopy) {
      RingPos pos;
      int issued = 0;
      bool ok = true;
      auto stream = [&](int r, bool last) {
        const T* src = logits + (size_t)r * p.ld + (size_t)v0 * E;
        for (int b = 0; b < nvec && ok; b += rs.stage) {
          if (!(ok = ring_wait(&bar.empty[pos.slot], pos.round ^ 1, p.status))) return;
          const uint32_t bytes = (uint32_t)min(rs.stage, nvec - b) * 16;
          tc::mbar_expect_tx(&bar.full[pos.slot], bytes);
          bulk_load(slots + (size_t)pos.slot * rs.stage, src + (size_t)b * E, bytes, &bar.full[pos.slot], last);
          pos.skip(1, rs.n_slots);
          issued++;
        }
      };
      float w = weight(cluster);
      bool live = false;
      for (int r = cluster; ok; r += n_clusters) {
        const int prev = r - n_clusters;
        if (kGrad ? prev >= p.n : r >= p.n) break;
        const float wn = weight(r + n_clusters);
        const bool was = live;
        live = r < p.n && w != 0.f;
        if (live) stream(r, !kGrad);
        if (kGrad && was) stream(prev, true);
        w = wn;
      }
      // a copy must not outlive the CTA: the consumers have seen all of them unless a wait gave up
      if (!ok)
        for (int i = min(issued, rs.n_slots); i > 0; i--) {
          if (--pos.slot < 0) pos.slot = rs.n_slots - 1, pos.round ^= 1;
          ring_wait(&bar.full[pos.slot], pos.round, p.status);
        }
    }
  } else if (tid >= kFirstCons) {
    // ---- consumers ----
    const int ct = tid - kFirstCons;
    const int group = ct / kGroupThreads, t = ct % kGroupThreads;
    const int n_st = (nvec + rs.stage - 1) / rs.stage, n_sub = rs.stage / kSub;
    // this group's next stage: its slot, and which of the next row's stages it is
    RingPos pos;
    pos.skip(group, rs.n_slots);
    int next = group;
    auto to_next_row = [&] { next = (next - n_st) & (kGroups - 1); };
    bool ok = true;
    StageStat<T, false> st;
    // sums over the entries outside the list
    auto sums = [&](int it, bool live) {
      const int b = it % kMaxRows;
      const uint32_t ph = it / kMaxRows & 1;
      st.init();
      float tm = -INFINITY;
      if (p.tail && !(ok = warp_wait(&bar.pre_full[b], ph, p.status))) return;
      if (live) {
        const uint32_t* bits = bitmap + b * p.words;
        for (int j = next; j < n_st; j += kGroups) {
          const int cnt = nvec - j * rs.stage;
          if (!(ok = warp_wait(&bar.full[pos.slot], pos.round, p.status))) return;
          const uint4* slot = slots + (size_t)pos.slot * rs.stage;
          for (int u = 0; u < n_sub; u++) {
            const int left = cnt - u * kSub;
            if (left <= 0) break;
            uint4 w[kPer];
            load_sub<T>(slot + u * kSub, left, t, w);
            if (p.tail) {
#pragma unroll
              for (int q = 0; q < kPer; q++) {
                const int i = q * kGroupThreads + (t & ~31);
                const uint32_t word = i < left ? bits[(j * rs.stage + u * kSub + i) >> 5] : 0;
                if (word >> lane & 1) w[q] = Raw<T>::masked();
              }
            }
            const float mx = Raw<T>::max(w);
            if (u + 1 == n_sub || left <= kSub) give_back(&bar.empty[pos.slot], mx);
            tm = fmaxf(tm, mx);
            st.add(w, left, mx, c2);
          }
          pos.skip(kGroups, rs.n_slots);
        }
        to_next_row();
      }
      Stat tot = st.total(tm, c2);
      warp_merge(tot, c2);
      if (!(ok = warp_wait(&bar.part_empty[b], ph ^ 1, p.status))) return;
      if (lane == 0) {
        ss.part[b][ct >> 5][0] = tot.m;
        ss.part[b][ct >> 5][1] = tot.s;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar.part_full[b]);
    };
    // the gradient of the entries outside the list (the listed ones are overwritten later)
    auto gradient = [&](int it, int r, bool live) {
      const int b = it % kMaxRows;
      if (!(ok = warp_wait(&bar.scal_full[b], it / kMaxRows & 1, p.status))) return;
      const RowScale sc = ss.scale[b];
      uint4* out = reinterpret_cast<uint4*>(dlogits + (size_t)r * p.ld) + v0;
      const f2 cc = pack2(c2, c2), hi = pack2(-sc.hi, -sc.hi), ff = pack2(sc.f, sc.f);
      for (int j = live ? next : group; j < n_st; j += kGroups) {
        const int cnt = min(rs.stage, nvec - j * rs.stage);
        if (live && !(ok = warp_wait(&bar.full[pos.slot], pos.round, p.status))) return;
        const uint4* slot = slots + (size_t)pos.slot * rs.stage;
        uint4* const dst = out + j * rs.stage;
        if (!sc.live) {
          for (int i = t; i < cnt; i += kGroupThreads) __stcs(dst + i, make_uint4(0, 0, 0, 0));
        } else if (sc.usual) {
#pragma unroll kPer
          for (int i = t; i < cnt; i += kGroupThreads) {
            const uint4 w = slot[i];
            float g[E];
#pragma unroll
            for (int e = 0; e < E / 2; e++) {
              float y0, y1;
              unpack2(fma2(Raw<T>::pair(w, e), cc, hi), y0, y1);
              unpack2(mul2(pack2(ex2f(y0), ex2f(y1)), ff), g[2 * e], g[2 * e + 1]);
            }
            __stcs(dst + i, VT::pack(g));
          }
        } else {
          for (int i = t; i < cnt; i += kGroupThreads) {
            float x[E], g[E];
            VT::cvt(slot[i], x);
#pragma unroll
            for (int e = 0; e < E; e++) g[e] = sc.f * ex2f(max_nan((x[e] - sc.m) * c2 - sc.l2, kCut));
            __stcs(dst + i, VT::pack(g));
          }
        }
        if (live) {
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bar.empty[pos.slot]);
          pos.skip(kGroups, rs.n_slots);
        }
      }
      if (live) to_next_row();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar.p2_done[b]);
    };
    float w = weight(cluster);
    bool live = false;
    for (int r = cluster, it = 0; ok; r += n_clusters, it++) {
      const int prev = r - n_clusters;
      if (kGrad ? prev >= p.n : r >= p.n) break;
      const float wn = weight(r + n_clusters);
      const bool was = live;
      live = r < p.n && w != 0.f;
      if (r < p.n) sums(it, live);
      if (kGrad && ok && it > 0) gradient(it - 1, prev, was);
      w = wn;
    }
  } else {
    // ---- finishers: the warps take the rows in turn ----
    const int b = tid >> 5;
    WarpSmem& ws = ss.warp[b];
    uint32_t* const bits = bitmap + b * p.words;
    const int tail_n = rank + 1 == (uint32_t)rs.cs ? p.V - nv * E : 0;
    const int step = kFinishers * n_clusters;
    // The lane's entries of the teacher's list (those from p.k on have no id), their
    // probabilities and logarithms, the sum of the list's probabilities of the same id, and
    // which entries are their id's first.
    int id[kEntries];
    float lp[kEntries], pe[kEntries], sub[kEntries];
    uint32_t first = 0;
    float w = 0.f, pr = 0.f, total = 0.f, last_x = 0.f;
    bool live = false, last_listed = false;
    Stat pre_o, pre_in;   // sums of the listed vectors and of the row's last entries
    int next_id[kEntries];
    float next_z[kEntries], next_w = 0.f;
    auto fetch = [&](int r) {
      if (r >= p.n) return;
      next_w = weight(r);
#pragma unroll
      for (int q = 0; q < kEntries; q++) {
        const int i = q * 32 + lane;
        next_id[q] = -1;
        if (i >= p.k) continue;
        next_id[q] = p.t_ids[(size_t)r * p.k + i];
        next_z[q] = p.t_val[(size_t)r * p.k + i];
      }
    };
    // What does not need the row's sums: the teacher's probabilities, which vectors hold listed
    // ids, and the sums over those vectors.  Its weight and entries were fetched a row earlier.
    auto prepare = [&](int r) {
      const T* row = logits + (size_t)r * p.ld;
      w = next_w;
      live = w != 0.f;
      first = 0;
      pre_o.init();
      pre_in.init();
      if (!live) {
        if (p.tail && lane == 0) tc::mbar_arrive(&bar.pre_full[b]);
        return;
      }
      float z[kEntries], x[kEntries];
#pragma unroll
      for (int q = 0; q < kEntries; q++) {
        id[q] = next_id[q];
        z[q] = next_z[q];
        if (id[q] >= p.V) atomicExch(p.status, OCTO_EINVAL);
        if (id[q] < 0 || id[q] >= p.V || z[q] == -INFINITY) id[q] = -1, z[q] = -INFINITY;
        x[q] = id[q] < 0 ? 0.f : VT::get(row + id[q]);
      }
      last_x = lane < tail_n ? VT::get(row + nv * E + lane) : -INFINITY;
      if (p.tail)
        for (int i = lane; i < p.words; i += 32) bits[i] = 0;
      float zm = -INFINITY, sum = 0.f;
#pragma unroll
      for (int q = 0; q < kEntries; q++) zm = fmaxf(zm, z[q]);
      zm = p.tail ? 0.f : warp_max(zm);
      total = 0.f;
#pragma unroll
      for (int q = 0; q < kEntries; q++) {
        lp[q] = z[q] == -INFINITY ? -INFINITY : p.tail ? z[q] : (z[q] - zm) * p.c;
        sum += expf(lp[q]);
      }
      sum = warp_sum(sum);
      const float ls = p.tail ? 0.f : logf(sum);
      if (!p.tail && sum == 0.f) live = false;   // no teacher
#pragma unroll
      for (int q = 0; q < kEntries; q++) {
        lp[q] -= ls;
        pe[q] = id[q] < 0 ? 0.f : expf(lp[q]);
        total += pe[q];
      }
      total = p.tail ? sum : warp_sum(total);
      pr = !p.tail ? 0.f : total != total ? total : fmaxf(0.f, 1.f - total);
      // Entries that share a vector, or an id, are few in general: a table of bits finds out
      // which may, and only those are compared with all the others.
      uint32_t mask[kEntries];   // listed ids in the entry's vector
      uint32_t first_vec = 0;
      uint32_t meets[kEntries];
#pragma unroll
      for (int i = 0; i < kHashWords; i += 32) ws.hash[i + lane] = 0;
      __syncwarp();
#pragma unroll
      for (int q = 0; q < kEntries; q++) {
        const uint32_t vec = (uint32_t)id[q] / E, h = (vec * 0x9e3779b1u) >> 21;
        const bool has_id = id[q] >= 0;
        sub[q] = pe[q];
        mask[q] = has_id ? 1u << ((uint32_t)id[q] % E) : 0u;
        first |= (uint32_t)has_id << q;
        first_vec |= (uint32_t)has_id << q;
        const bool hit = has_id && (atomicOr(&ws.hash[h / 32], 1u << h % 32) >> h % 32 & 1);
        meets[q] = __ballot_sync(0xffffffffu, hit);
      }
      uint32_t shares = 0;       // bit q: another entry is in this one's vector
#pragma unroll
      for (int q = 0; q < kEntries; q++)
        for (uint32_t left = meets[q]; left; left &= left - 1) {
          const int l = __ffs(left) - 1;
          const uint32_t vec = (uint32_t)__shfl_sync(0xffffffffu, id[q], l) / E;
          uint32_t with = 0;
#pragma unroll
          for (int q2 = 0; q2 < kEntries; q2++)
            with |= (uint32_t)((uint32_t)id[q2] / E == vec && !(q2 == q && l == lane)) << q2;
          shares |= with;
          if (__any_sync(0xffffffffu, with != 0) && l == lane) shares |= 1u << q;
        }
#pragma unroll
      for (int q = 0; q < kEntries; q++)   // in the entries' order, so that the sums are always the same
        for (uint32_t left = __ballot_sync(0xffffffffu, shares >> q & 1); left; left &= left - 1) {
          const int l = __ffs(left) - 1;
          const uint32_t other = __shfl_sync(0xffffffffu, id[q], l);
          const float po = __shfl_sync(0xffffffffu, pe[q], l);
#pragma unroll
          for (int q2 = 0; q2 < kEntries; q2++) {
            const bool self = q2 == q && l == lane, before = q < q2 || (q == q2 && l < lane);
            const bool same_vec = other / E == (uint32_t)id[q2] / E && !self, same_id = other == (uint32_t)id[q2] && !self;
            if (same_vec) mask[q2] |= 1u << (other % E);
            if (same_id) sub[q2] += po;
            if (same_vec && before) first_vec &= ~(1u << q2);
            if (same_id && before) first &= ~(1u << q2);
          }
        }
      uint32_t listed = 0;   // of the last entries
      if (tail_n > 0) {
#pragma unroll
        for (int q = 0; q < kEntries; q++)
          if (id[q] >= nv * E) listed |= 1u << (id[q] - nv * E);
        listed = __reduce_or_sync(0xffffffffu, listed);
      }
      last_listed = listed >> lane & 1;
      if (p.tail) {
#pragma unroll
        for (int q = 0; q < kEntries; q++) {
          const int vec = id[q] / E, at = vec - v0;
          if (!(first_vec >> q & 1) || vec < v0 || at >= nvec) continue;
          atomicOr(&bits[at >> 5], 1u << (at & 31));
          float y[E];
          VT::cvt(reinterpret_cast<const uint4*>(row)[vec], y);
          float mo = pre_o.m, mi = pre_in.m;
#pragma unroll
          for (int e = 0; e < E; e++) (mask[q] >> e & 1 ? mi : mo) = fmaxf(mask[q] >> e & 1 ? mi : mo, y[e]);
          pre_o.rebase(mo, c2);
          pre_in.rebase(mi, c2);
#pragma unroll
          for (int e = 0; e < E; e++) {
            const bool in = mask[q] >> e & 1;
            const float x2 = ex2f(max_nan((y[e] - (in ? mi : mo)) * c2, kCut));
            (in ? pre_in.s : pre_o.s) += x2;
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar.pre_full[b]);
      }
      if (lane < tail_n) {
        Stat s{fmaxf(last_x, -FLT_MAX), 0.f, 0.f};
        s.add(last_x, c2);
        if (p.tail && last_listed) pre_in.merge(s.m, s.s, 0.f, c2);
        else pre_o.merge(s.m, s.s, 0.f, c2);
      }
      if (p.tail || tail_n > 0) warp_merge(pre_o, c2);
      if (p.tail) warp_merge(pre_in, c2);
      // waits for the loads: a peer may overwrite the row once it has this CTA's sums
#pragma unroll
      for (int q = 0; q < kEntries; q++) ws.x[q * 32 + lane] = x[q];
    };
    const int first_row = cluster + b * n_clusters;
    fetch(first_row);
    if (first_row < p.n) prepare(first_row);
    for (int r = first_row, turn = 0; r < p.n; r += step, turn++) {
      const uint32_t ph = turn & 1;
      fetch(r + step);
      if (!warp_wait(&bar.part_full[b], ph, p.status)) break;
      Stat o = pre_o, in = pre_in;
      if (live) {
        Stat s;
        s.init();
        if (lane < kConsWarps) s.m = ss.part[b][lane][0], s.s = ss.part[b][lane][1];
        warp_merge(s, c2);
        o.merge(s.m, s.s, 0.f, c2);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar.part_empty[b]);
      if (rs.cs > 1) {
        // every CTA to every CTA; in[] and the barriers by turns, so that a fast CTA's next row
        // meets nobody who still reads or waits for this one
        uint64_t* const joined = &bar.joined[b][ph];
        if (lane == 0) tc::mbar_expect_tx(joined, rs.cs * 16);
        if (lane < rs.cs)
          st_async(map_rank(tc::smem_u32(ws.in[ph][rank]), lane), o.m, o.s, in.m, in.s, map_rank(tc::smem_u32(joined), lane));
        if (!__all_sync(0xffffffffu, ring_wait<true>(joined, turn >> 1 & 1, p.status))) break;
        o.init();
        in.init();
        if (lane < rs.cs) {
          const float* q = ws.in[ph][lane];
          o.m = q[0], o.s = q[1], in.m = q[2], in.s = q[3];
        }
        warp_merge(o, c2);
        if (p.tail) warp_merge(in, c2);
      }
      Stat all = o;
      if (p.tail) all.merge(in.m, in.s, 0.f, c2);
      const bool has = live && all.s != 0.f;
      const float f = p.gs * w * p.c;
      float ls = 0.f, ls_lo = 0.f, lqr = 0.f, qr = 0.f;
      RowScale sc = {0.f, 0.f, 0.f, 0.f, 0, 1};
      if (has) {
        const float lo = logf(o.s);
        split_log(all.s, &ls, &ls_lo);
        sc.live = 1;
        if (!p.tail) {
          sc.f = f * total;
        } else if (o.s == 0.f || (o.m - all.m) * p.c - ls < kNoMass) {
          pr = 0.f;   // nothing outside the list has mass (o's sum is relative to its own largest entry)
        } else {
          // ln q_R: by the ratio of the sums, unless one's reference is too far below the other's
          Stat far = o;
          far.rebase(all.m, c2);
          lqr = far.s > 1e-30f ? logf(far.s / all.s) : (o.m - all.m) * p.c + lo - ls - ls_lo;
          qr = expf(lqr);
          sc.f = f * (qr * (total + pr) - pr);
        }
        if (o.s != 0.f) sc.m = o.m, sc.l2 = lo * kLog2e;
        sc.usual = StageStat<T, false>::usual(sc.m, c2);
        // hi = c2 m + l2 rounded; what it leaves out goes into the factor.  Each operation rounded
        // by itself: a product fused into the difference after it would count its error twice.
        const float a = __fmul_rn(sc.m, c2), ae = fmaf(sc.m, c2, -a);
        sc.hi = __fadd_rn(a, sc.l2);
        const float d = __fsub_rn(sc.hi, a);
        if (sc.usual) sc.f *= ex2f(-(ae + (__fsub_rn(a, __fsub_rn(sc.hi, d)) + __fsub_rn(sc.l2, d))));
      }
      if (kGrad && lane == 0) {
        ss.scale[b] = sc;
        tc::mbar_arrive(&bar.scal_full[b]);
      }
      float kl = 0.f, fix[kEntries];
#pragma unroll
      for (int q = 0; q < kEntries; q++) {
        fix[q] = 0.f;
        if (!has || id[q] < 0) continue;
        const float lq = fmaf(ws.x[q * 32 + lane] - all.m, p.c, -ls) - ls_lo;
        if (first >> q & 1) {   // an id's entries are one class, its first one's
          const float P = sub[q], d = (P == pe[q] ? lp[q] : logf(P)) - lq;
          if (p.tail) kl += share(P, d, expf(lq));
          else if (P != 0.f) kl += P * d;
        }
        if (kGrad) fix[q] = f * (expf(lq) * (total + pr) - sub[q]);
      }
      if (rank == 0) {
        kl = warp_sum(kl);
        if (has && p.tail)   // without a rest in the teacher its masses need not be 1 in sum
          kl += pr != 0.f ? share(pr, logf(pr) - lqr, qr) : qr + (total - 1.f);
        if (lane == 0) {
          p.row_kl[p.row0 + r] = kl;
          if (p.part) p.part[r] = has ? w * kl : 0.f;
        }
      }
      int fixed[kEntries];   // the ids that this lane writes: firsts, in this CTA's part
#pragma unroll
      for (int q = 0; q < kEntries; q++) {
        const int vec = id[q] / E;
        const bool own = vec < nv ? vec >= v0 && vec < v0 + nvec : tail_n > 0;
        fixed[q] = has && (first >> q & 1) && own ? id[q] : -1;
      }
      const float done_x = last_x;
      const bool done_listed = has && last_listed;
      if (r + step < p.n) prepare(r + step);
      if (kGrad) {
        // after the consumers' stores: the listed entries, each id by its first, and the last ones
        if (!warp_wait(&bar.p2_done[b], ph, p.status)) break;
        T* grow = dlogits + (size_t)r * p.ld;
#pragma unroll
        for (int q = 0; q < kEntries; q++)
          if (fixed[q] >= 0) VT::put(grow + fixed[q], fix[q]);
        if (lane < tail_n && !done_listed)
          VT::put(grow + nv * E + lane, sc.live ? sc.f * ex2f(sc.usual ? fmaf(done_x, c2, -sc.hi)
                                                                         : max_nan((done_x - sc.m) * c2 - sc.l2, kCut))
                                                 : 0.f);
      }
    }
  }
  // no CTA leaves while another may still write to its shared memory
  __syncwarp();
  if (rs.cs > 1) cluster_sync();
}

template <typename T>
int launch_distill(DistillParams& p, cudaStream_t s) {
  const int64_t nv = p.V / Vec<T>::E;
  const void* f = p.dlogits ? (p.k <= 32   ? (const void*)k_distill<T, true, 1>
                               : p.k <= 64 ? (const void*)k_distill<T, true, 2>
                                           : (const void*)k_distill<T, true, 4>)
                            : (p.k <= 32   ? (const void*)k_distill<T, false, 1>
                               : p.k <= 64 ? (const void*)k_distill<T, false, 2>
                                           : (const void*)k_distill<T, false, 4>);
  auto words = [&](int cs) { return (int)(((nv + cs - 1) / cs + 31) / 32); };
  int cs = 1;
  if (int st = pick_cluster(f, p.n, p.dlogits ? 2 * nv : nv, kSmemMax, [](int) { return 0.7; }, &cs)) return st;
  if (p.dlogits && cs == 1) {
    // Two rows for each cluster wait in L2 for their second pass, and their gradients pass
    // through it: past three tenths of it they are read from memory again.  More CTAs a row
    // mean fewer rows in flight, at the price of joining the CTAs at every row, and want rows
    // for several rounds.  Microseconds at 1 / 2 / 4 CTAs, bf16 rows of 64 entries, 4,000 of
    // them (3,000 from 350 KB on, 2,000 of 608 KB), without and with the rest class:
    //   128 KB (29 % of L2 at 1 CTA)  176 / 198 / 287   174 / 210 / 343
    //   160 KB (37 %)                 226 / 205 / 302   229 / 219 / 343
    //   200 KB (46 %)                 293 / 253 / 358   299 / 262 / 383
    //   250 KB (58 %)                 395 / 320 / 398   402 / 318 / 430
    //   304 KB (70 %)                 501 / 407 / 382   512 / 401 / 430
    //   350 KB (81 %)                 440 / 370 / 335   448 / 374 / 368
    //   400 KB (92 %)                 504 / 440 / 370   513 / 446 / 394
    //   608 KB (140 %)                520 / 501 / 380   531 / 510 / 387
    // fp32 rows, with half the entries, like four CTAs earlier: 160 KB 226 / 209 / 261 and
    // 228 / 208 / 280, 240 KB 366 / 312 / 364 and 376 / 309 / 379, 304 KB 493 / 415 / 366 and
    // 500 / 411 / 375.  So a row gets two CTAs, and four, past three tenths, but bf16 rows with
    // the rest class, whose CTAs each clear and fill a bitmap, get four past four tenths.
    const int sms = sm_count();
    auto in_flight = [&](int c) { return (int64_t)nv * 16 * 2 * (sms / c); };
    auto room = [&](int c) { return l2_bytes() / 100 * (c == 2 && p.tail && Vec<T>::E == 8 ? 40 : 30); };
    while (cs < 4 && in_flight(cs) > room(cs) && (int64_t)p.n * 2 * cs > 5 * sms) cs *= 2;
  }
  while (words(cs) * 4 * kMaxRows > 64 * 1024 && cs < kMaxCluster) cs *= 2;
  p.words = p.tail ? words(cs) : 0;
  p.ring = ring_shape(nv, cs, kSmemMax - slots_offset(p.words));
  if (p.ring.n_slots < kGroups) return OCTO_ENOTSUP;
  return launch_ring(f, p, p.n, cs, slots_offset(p.words) + p.ring.n_slots * p.ring.stage * 16, s);
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
  if (!teach_ids || !teach_val || !row_kl || (loss && (!ws || ws_bytes < need || ((uintptr_t)ws & 3)))) return OCTO_EINVAL;
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
  p.n = n_rows;
  if (int st = dtype == OCTO_DTYPE_BF16 ? launch_distill<__nv_bfloat16>(p, s) : launch_distill<float>(p, s)) return st;
  return loss ? launch_loss_sum((const float*)ws, n_rows, loss, s) : OCTO_OK;
}

}  // extern "C"
