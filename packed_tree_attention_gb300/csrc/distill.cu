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
// What the listed entries need: the reference and logarithm of the whole sum, the teacher's
// rest and the logarithm of the student's.
struct RowSums {
  float m, ls, pr, lqr;
  int32_t has;
};
struct __align__(16) TeamSmem {
  int32_t id[kMaxTop];
  __align__(16) int32_t vec[kMaxTop];   // vectors of the ids
  float p[kMaxTop], x[kMaxTop];
  uint32_t last;                       // listed ones of the row's last entries
  float red[2][kFinWarps];
  float pre_o[kFinWarps][2], pre_in[kFinWarps][2];   // sums of the listed vectors and of the last entries
  RowSums res[2];                                    // by turns
  __align__(16) float in[2][kMaxCluster][4];                       // the CTAs' sums, of every other row of the team
};
struct DistillSmem {
  RingBars bars;
  float part[2][kConsWarps][2];
  RowScale scale[2];
  TeamSmem team[kTeams];
};
constexpr int kBitmapOffset = ((int)sizeof(DistillSmem) + 127) / 128 * 128;
__host__ __device__ constexpr int slots_offset(int words) { return kBitmapOffset + (kTeams * words * 4 + 127) / 128 * 128; }

__device__ __forceinline__ float fin_fold(float v, TeamSmem& t, int team, int& buf) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int w = ((int)threadIdx.x - team * kFin) >> 5;
  if ((threadIdx.x & 31) == 0) t.red[buf][w] = v;
  fin_sync(team);
  float r = 0.f;
#pragma unroll
  for (int i = 0; i < kFinWarps; i++) r += t.red[buf][i];
  buf ^= 1;
  return r;
}
__device__ __forceinline__ float fin_max(float v, TeamSmem& t, int team, int& buf) {
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(v) : "f"(v));
  const int w = ((int)threadIdx.x - team * kFin) >> 5;
  if ((threadIdx.x & 31) == 0) t.red[buf][w] = v;
  fin_sync(team);
  float r = t.red[buf][0];
#pragma unroll
  for (int i = 1; i < kFinWarps; i++) r = fmaxf(r, t.red[buf][i]);
  buf ^= 1;
  return r;
}

// A finisher thread's entry of the teacher's list, made ready before the row's sums.
struct Entry {
  int id = -1;       // -1: none
  float lp = 0.f, p = 0.f, x = 0.f;
  float sub = 0.f;   // sum of the list's probabilities of this id
  bool first = false;   // the id's first entry
};

// With a gradient every row is streamed twice, the first pass of the next row before the second
// of this one, so that the join of the row's sums is not waited for.  The second time a row
// comes from L2 (two rows for each cluster in flight).
template <typename T, bool kGrad>
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

  if (tid == 0) bar.init();
  __syncthreads();
  if (rs.cs > 1) cluster_sync();

  if (tid >= kCopy && tid < kFirstCons) {
    // ---- copies (rows of weight 0 are not read) ----
    if (tid == kCopy) {
      RingPos pos;
      int issued = 0;
      bool ok = true;
      auto stream = [&](int r) {
        const T* src = logits + (size_t)r * p.ld + (size_t)v0 * E;
        for (int b = 0; b < nvec && ok; b += rs.stage) {
          if (!(ok = ring_wait(&bar.empty[pos.slot], pos.round ^ 1, p.status))) return;
          const uint32_t bytes = (uint32_t)min(rs.stage, nvec - b) * 16;
          tc::mbar_expect_tx(&bar.full[pos.slot], bytes);
          bulk_load(slots + (size_t)pos.slot * rs.stage, src + (size_t)b * E, bytes, &bar.full[pos.slot]);
          pos.skip(1, rs.n_slots);
          issued++;
        }
      };
      float w = weight(cluster), was = 0.f;
      for (int r = cluster; r - n_clusters < p.n && ok; r += n_clusters) {
        const float wn = weight(r + n_clusters);
        if (r < p.n && w != 0.f) stream(r);
        if (kGrad && was != 0.f) stream(r - n_clusters);
        was = w;
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
      const int par = it & 1;
      const uint32_t ph = (it >> 1) & 1;
      st.init();
      float tm = -INFINITY;
      if (p.tail && !(ok = warp_wait(&bar.pre_full[par], ph, p.status))) return;
      if (live) {
        const uint32_t* bits = bitmap + par * p.words;
        for (int j = next; j < n_st; j += kGroups) {
          const int cnt = nvec - j * rs.stage;
          if (!(ok = warp_wait(&bar.full[pos.slot], pos.round, p.status))) return;
          const uint4* slot = slots + (size_t)pos.slot * rs.stage;
          for (int u = 0; u < n_sub; u++) {
            const int left = cnt - u * kSub;
            if (left <= 0) break;
            uint4 w[kPer];
            load_sub<T>(slot + u * kSub, left, t, w);
            if (u + 1 == n_sub || left <= kSub) {
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&bar.empty[pos.slot]);
            }
            if (p.tail) {
#pragma unroll
              for (int q = 0; q < kPer; q++) {
                const int i = q * kGroupThreads + (t & ~31);
                const uint32_t word = i < left ? bits[(j * rs.stage + u * kSub + i) >> 5] : 0;
                if (word >> lane & 1) w[q] = Raw<T>::masked();
              }
            }
            const float mx = Raw<T>::max(w);
            tm = fmaxf(tm, mx);
            st.add(w, left, mx, c2);
          }
          pos.skip(kGroups, rs.n_slots);
        }
        to_next_row();
      }
      Stat tot = st.total(tm, c2);
      warp_merge(tot, c2);
      if (!(ok = warp_wait(&bar.part_empty[par], ph ^ 1, p.status))) return;
      if (lane == 0) {
        ss.part[par][ct >> 5][0] = tot.m;
        ss.part[par][ct >> 5][1] = tot.s;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar.part_full[par]);
    };
    // the gradient of the entries outside the list (the listed ones are overwritten later)
    auto gradient = [&](int it, int r, bool live) {
      const int par = it & 1;
      if (!(ok = warp_wait(&bar.scal_full[par], (it >> 1) & 1, p.status))) return;
      const RowScale sc = ss.scale[par];
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
      if (lane == 0) tc::mbar_arrive(&bar.p2_done[par]);
    };
    float w = weight(cluster);
    bool live = w != 0.f, was = false;
    for (int r = cluster, it = 0; ok; r += n_clusters, it++) {
      const float wn = weight(r + n_clusters);
      if (r < p.n) sums(it, live);
      if (kGrad && ok && it > 0) gradient(it - 1, r - n_clusters, was);
      if (r >= p.n) break;
      was = live;
      live = wn != 0.f;
    }
  } else {
    // ---- finishers: team `par` takes the rows of that parity ----
    const int par = tid / kFin, ft = tid - par * kFin, wi = ft >> 5;
    TeamSmem& ts = ss.team[par];
    uint32_t* const bits = bitmap + par * p.words;
    const int tail_n = rank + 1 == (uint32_t)rs.cs ? p.V - nv * E : 0;
    int buf = 0;
    // what does not need the row's sums: the teacher's probabilities, which vectors hold listed
    // ids, and the sums over those vectors and the row's last entries.  A row that is not live
    // has none of it.
    Entry en;
    float w = 0.f, pr = 0.f, total = 0.f, tail_x = 0.f;
    bool live = false, tail_listed = false;
    // its weight and entries are fetched a row earlier
    int next_id = -1;
    float next_z = 0.f, next_w = 0.f;
    auto fetch = [&](int r) {
      if (r >= p.n) return;
      next_w = weight(r);
      if (ft < p.k) {
        next_id = p.t_ids[(size_t)r * p.k + ft];
        next_z = p.t_val[(size_t)r * p.k + ft];
      }
    };
    auto prepare = [&](int r) {
      const T* row = logits + (size_t)r * p.ld;
      en = Entry();
      w = next_w;
      live = w != 0.f;
      float z = -INFINITY;
      if (live && ft < p.k) {
        en.id = next_id;
        z = next_z;
        if (en.id >= p.V) atomicExch(p.status, OCTO_EINVAL);
        if (en.id < 0 || en.id >= p.V || z == -INFINITY) en.id = -1, z = -INFINITY;
      }
      const int vec = en.id < 0 ? -1 : en.id / E;
      const bool own = vec >= v0 && vec < v0 + nvec;
      uint4 wv = make_uint4(0, 0, 0, 0);
      if (en.id >= 0) en.x = VT::get(row + en.id);
      if (p.tail && own) wv = reinterpret_cast<const uint4*>(row)[vec];
      tail_x = live && ft < tail_n ? VT::get(row + nv * E + ft) : -INFINITY;
      if (!live) {
        if (p.tail) {
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bar.pre_full[par]);
        }
        fin_sync(par);
        return;
      }
      ts.id[ft] = en.id;
      ts.vec[ft] = vec;
      if (ft == 0) ts.last = 0;
      if (p.tail) {
        for (int i = ft; i < p.words; i += kFin) bits[i] = 0;
        en.lp = z;
        en.p = expf(z);
        total = fin_fold(en.p, ts, par, buf);
        pr = total != total ? total : fmaxf(0.f, 1.f - total);
      } else {
        const float zm = fin_max(z, ts, par, buf);
        const float t = z == -INFINITY ? -INFINITY : (z - zm) * p.c;
        const float sum = fin_fold(expf(t), ts, par, buf);
        pr = 0.f;
        if (sum == 0.f) live = false;   // no teacher
        en.lp = t - logf(sum);
        en.p = en.id < 0 ? 0.f : expf(en.lp);
        total = fin_fold(en.p, ts, par, buf);
      }
      ts.p[ft] = en.p;
      if (vec == nv) atomicOr(&ts.last, 1u << (en.id % E));
      fin_sync(par);
      Stat o, in;
      o.init();
      in.init();
      if (en.id >= 0) {
        uint32_t mask = 1u << (en.id % E);
        bool first_vec = true;
        en.sub = en.p;
        en.first = true;
        auto same = [&](int i) {   // another entry in this one's vector
          const int other = ts.id[i];
          mask |= 1u << (other % E);
          first_vec = first_vec && i > ft;
          if (other == en.id) en.sub += ts.p[i], en.first = en.first && i > ft;
        };
        for (int i = 0; i < p.k; i += 4) {   // entries past k have vec -1
          const int4 o4 = *reinterpret_cast<const int4*>(&ts.vec[i]);
          const bool x = o4.x == vec && i != ft, y = o4.y == vec && i + 1 != ft, z4 = o4.z == vec && i + 2 != ft,
                     w4 = o4.w == vec && i + 3 != ft;
          if (x || y || z4 || w4) {
            if (x) same(i);
            if (y) same(i + 1);
            if (z4) same(i + 2);
            if (w4) same(i + 3);
          }
        }
        if (p.tail && own && first_vec) {
          const int at = vec - v0;
          atomicOr(&bits[at >> 5], 1u << (at & 31));
          float x[E];
          VT::cvt(wv, x);
#pragma unroll
          for (int e = 0; e < E; e++) {
            Stat& s = mask >> e & 1 ? in : o;
            if (x[e] > s.m) s.rebase(x[e], c2);
            s.add(x[e], c2);
          }
        }
      }
      if (p.tail) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar.pre_full[par]);
      }
      tail_listed = false;
      if (ft < tail_n) {
        tail_listed = ts.last >> ft & 1;
        Stat& s = p.tail && tail_listed ? in : o;
        if (tail_x > s.m) s.rebase(tail_x, c2);
        s.add(tail_x, c2);
      }
      if (p.tail || tail_n > 0) warp_merge(o, c2);
      if (p.tail) warp_merge(in, c2);
      if (lane == 0) {
        ts.pre_o[wi][0] = o.m, ts.pre_o[wi][1] = o.s;
        ts.pre_in[wi][0] = in.m, ts.pre_in[wi][1] = in.s;
      }
      ts.x[ft] = en.x;   // waits for the load: a peer may overwrite the row once it has this CTA's sums
      fin_sync(par);
    };
    const int first_row = cluster + par * n_clusters;
    fetch(first_row);
    if (first_row < p.n) prepare(first_row);
    for (int r = first_row, it = par; r < p.n; r += 2 * n_clusters, it += 2) {
      const uint32_t ph = (it >> 1) & 1;
      fetch(r + 2 * n_clusters);
      bool ok = true;
      if (wi == 0) {
        // the row's sums and what the gradient pass needs of them, by one warp: the consumers
        // wait for it
        ok = warp_wait(&bar.part_full[par], ph, p.status);
        Stat o, in;
        o.init();
        in.init();
        if (ok && live) {
          if (lane < kConsWarps) o.m = ss.part[par][lane][0], o.s = ss.part[par][lane][1];
          else if (lane < kConsWarps + kFinWarps) o.m = ts.pre_o[lane - kConsWarps][0], o.s = ts.pre_o[lane - kConsWarps][1];
          warp_merge(o, c2);
          if (p.tail) {
            if (lane < kFinWarps) in.m = ts.pre_in[lane][0], in.s = ts.pre_in[lane][1];
            warp_merge(in, c2);
          }
        }
        if (ok && rs.cs > 1) {
          // every CTA to every CTA; in[] and the barriers by turns, so that a fast CTA's next
          // row meets nobody who still reads or waits for this one
          uint64_t* const joined = &bar.joined[par][ph];
          if (lane == 0) tc::mbar_expect_tx(joined, rs.cs * 16);
          if (lane < rs.cs)
            st_async(map_rank(tc::smem_u32(ts.in[ph][rank]), lane), o.m, o.s, in.m, in.s, map_rank(tc::smem_u32(joined), lane));
          ok = __all_sync(0xffffffffu, ring_wait<true>(joined, (it >> 2) & 1, p.status));
          o.init();
          in.init();
          if (lane < rs.cs) {
            const float* q = ts.in[ph][lane];
            o.m = q[0], o.s = q[1], in.m = q[2], in.s = q[3];
          }
          warp_merge(o, c2);
          if (p.tail) warp_merge(in, c2);
        }
        Stat all = o;
        if (p.tail) all.merge(in.m, in.s, 0.f, c2);
        RowSums res = {all.m, 0.f, 0.f, 0.f, 0};
        RowScale sc = {0.f, 0.f, 0.f, 0.f, 0, 1};
        if (live && all.s != 0.f) {
          const float lo = logf(o.s);
          res.has = 1;
          res.ls = logf(all.s);
          res.pr = o.s == 0.f ? 0.f : pr;   // dropped where nothing outside the list has mass
          res.lqr = (o.m - all.m) * p.c + lo - res.ls;
          const float f = p.gs * w * p.c;
          sc.live = 1;
          sc.f = o.s == 0.f ? 0.f : f * (p.tail ? expf(res.lqr) * (total + res.pr) - res.pr : total);
          if (o.s != 0.f) sc.m = o.m, sc.l2 = lo * kLog2e;
          sc.usual = StageStat<T, false>::usual(sc.m, c2);
          // hi = c2 m + l2 rounded; what it leaves out goes into the factor
          const float a = sc.m * c2, ae = fmaf(sc.m, c2, -a);
          sc.hi = a + sc.l2;
          const float b = sc.hi - a;
          if (sc.usual) sc.f *= ex2f(-(ae + ((a - (sc.hi - b)) + (sc.l2 - b))));
        }
        if (lane == 0) {
          if (kGrad) {
            ss.scale[par] = sc;
            tc::mbar_arrive(&bar.scal_full[par]);
          }
          ts.res[ph] = res;
        }
      }
      if (!fin_all(ok, par)) break;
      if (lane == 0) tc::mbar_arrive(&bar.part_empty[par]);
      const RowSums res = ts.res[ph];
      const bool has = res.has;
      float fix = 0.f;
      if (has) {
        const float lq = en.id >= 0 ? (en.x - res.m) * p.c - res.ls : 0.f;
        if (rank == 0) {
          float kl = fin_fold(en.p != 0.f ? en.p * (en.lp - lq) : 0.f, ts, par, buf);
          if (res.pr != 0.f) kl += res.pr * (logf(res.pr) - res.lqr);
          if (ft == 0) {
            p.row_kl[p.row0 + r] = kl;
            if (p.part) p.part[r] = w * kl;
          }
        }
        fix = p.gs * w * p.c * (expf(lq) * (total + res.pr) - en.sub);
      } else if (rank == 0 && ft == 0) {
        p.row_kl[p.row0 + r] = 0.f;
        if (p.part) p.part[r] = 0.f;
      }
      const Entry done = en;
      const float last_x = tail_x;
      const bool last_listed = tail_listed;
      if (r + 2 * n_clusters < p.n) prepare(r + 2 * n_clusters);
      if (kGrad) {
        // after the consumers' stores: the listed entries, each id by its first, and the last ones
        if (!fin_all(ring_wait(&bar.p2_done[par], ph, p.status), par)) break;
        T* grow = dlogits + (size_t)r * p.ld;
        if (has && done.id >= 0 && done.first) {
          const int vec = done.id / E;
          if (vec < nv ? vec >= v0 && vec < v0 + nvec : tail_n > 0) VT::put(grow + done.id, fix);
        }
        const RowScale& sc = ss.scale[par];   // written again after the team's next row
        if (ft < tail_n && !(has && last_listed))
          VT::put(grow + nv * E + ft, sc.live ? sc.f * ex2f(sc.usual ? fmaf(last_x, c2, -sc.hi)
                                                                      : max_nan((last_x - sc.m) * c2 - sc.l2, kCut))
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
  const void* f = p.dlogits ? (const void*)k_distill<T, true> : (const void*)k_distill<T, false>;
  auto words = [&](int cs) { return (int)(((nv + cs - 1) / cs + 31) / 32); };
  int cs = 1;
  if (int st = pick_cluster(f, p.n, p.dlogits ? 2 * nv : nv, kSmemMax, [](int) { return 0.7; }, &cs)) return st;
  while (words(cs) * 4 * kTeams > 64 * 1024 && cs < kMaxCluster) cs *= 2;
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
  p.n = n_rows;
  if (int st = dtype == OCTO_DTYPE_BF16 ? launch_distill<__nv_bfloat16>(p, s) : launch_distill<float>(p, s)) return st;
  return loss ? launch_loss_sum((const float*)ws, n_rows, loss, s) : OCTO_OK;
}

}  // extern "C"
