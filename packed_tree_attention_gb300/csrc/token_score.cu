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
//
// Bound by memory: scoring reads V entries, the gradient reads and writes V.  Measured (one
// GB300, 6.78 TB/s copied): 10,240 rows of 151,936 bf16 scored in 430 us (7.2 TB/s), 2,048 rows
// with their top 64 in 119 us (5.2 TB/s: 13.5 rows an SM take 14 rounds, and the last row's
// alternatives follow its sums), 256 rows with their top 20 in 23 us (two rounds), one row in
// 11 us, most of it the chain from the launch over the copies, the threshold and the candidates
// to the join of the cluster.  The gradient of 6,144 such rows takes 545 us (6.8 TB/s).

#include <algorithm>

#include "row_ring.cuh"

namespace octo {
namespace {

using namespace rows;

constexpr int kFinWarps = 4, kFin = kFinWarps * 32;   // a team of finishers
constexpr int kTeams = kFinishers / kFinWarps;
constexpr int kFinBar = 1;           // named barriers of the teams: this and the next
static_assert(kTeams == 2, "team = parity of the row");
static_assert(kFin >= kMaxTop, "a thread for each alternative");
constexpr int kMaxBins = 10;         // bins of a thread's vectors
constexpr int kMaxCand = 1280, kMaxHits = 512, kMaxTrim = 512;
static_assert(kMaxCand >= kMaxCluster * kMaxTop, "the CTAs' alternatives are joined in cand");

struct ScoreParams {
  const void* logits;
  int64_t ld;
  int32_t V, row0, n, k;
  float c;
  const int32_t* ids;    // [plan rows] or null
  float* logp;           // [plan rows] or null
  float* row_stat;       // [n][2]
  float* entropy;        // [n] or null
  int32_t* top_ids;      // [n][k]
  float* top_logp;       // [n][k]
  SuccTable succ;
  int32_t* status;
  RingShape ring;
  // A thread's vectors, kPer at a time in `subs` turns at most, fall into `bins` bins.
  int32_t subs, bins;
};

// The first of a CTA's n_st stages of its row `it` that is the group's: the groups take the
// stages in turn, on over row ends.
__device__ __forceinline__ int first_stage(int group, int it, int n_st) {
  return (int)((uint32_t)group - (uint32_t)it * (uint32_t)n_st) & (kGroups - 1);
}

// Shared memory of the finishers; the ring's slots follow.
struct ScoreSmem {
  RingBars bars;
  float part[2][kConsWarps][3];          // a row's warp sums
  __align__(16) float in_stat[kMaxCluster][4];   // rank 0: the CTAs' sums
  float stat[2][2];                      // a row's (m, ln S), for the look-ups
};
// One of each for the two finisher teams.
struct TopSmem {
  unsigned long long in_list[kMaxCluster][kMaxTop];   // rank 0: the CTAs' alternatives, best first
  unsigned long long cand[kMaxCand];
  unsigned long long trim[kMaxTrim];
  unsigned long long sorted[kMaxTop];
  uint16_t hit[kMaxHits];
  uint32_t red[2][kFinWarps];
  int32_t n_hits, n_cand, n_ties, n_trim;
  float bmax[kMaxBins][kCons];           // largest entry of each bin of each thread's vectors
  float tmax[kCons];                     // and of each thread
};

template <bool kTop>
__host__ __device__ constexpr int ring_offset() {
  return (((int)sizeof(ScoreSmem) + 15) / 16 * 16 + (kTop ? kTeams * (int)sizeof(TopSmem) : 0) + 127) / 128 * 128;
}

// An alternative: the value's key above the complement of its id, so that among equal values
// the lowest id is the largest.
__device__ __forceinline__ unsigned long long cand_of(uint32_t key, int32_t v) {
  return ((unsigned long long)key << 32) | (uint32_t)~v;
}

__device__ __forceinline__ void fin_sync(int team) { asm volatile("bar.sync %0, %1;" ::"r"(kFinBar + team), "n"(kFin) : "memory"); }
// Uniform over the team: after a wait that gave up, all of it leaves together and none is left at
// a barrier.
__device__ __forceinline__ bool fin_all(bool ok, int team) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"((uint32_t)ok), "r"(kFinBar + team), "n"(kFin)
      : "memory");
  return all != 0;
}
__device__ __forceinline__ int fin_thread(int team) { return (int)threadIdx.x - team * kFin; }

// Sum over the finishers; red is used alternately (buf) so that one barrier is enough.
__device__ __forceinline__ uint32_t fin_sum(uint32_t v, TopSmem& ts, int team, int& buf) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) ts.red[buf][fin_thread(team) >> 5] = v;
  fin_sync(team);
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < kFinWarps; i++) r += ts.red[buf][i];
  buf ^= 1;
  return r;
}

// The k best of the n_cand candidates into ts.sorted, best first; returns how many.  At least
// k of them (or all) reach the key `lo`.  A candidate's rank is counted; where there are many,
// those below a lower bound of the k-th go first, found by a bisection.
__device__ int rank_cand(TopSmem& ts, int team, int k, uint32_t lo, int& buf) {
  const int ft = fin_thread(team);
  int n = ts.n_cand;
  const unsigned long long* from = ts.cand;
  if (n > 2 * kFin) {
    uint32_t hi = 0;
    for (int i = ft; i < n; i += kFin) hi = max(hi, (uint32_t)(ts.cand[i] >> 32));
    hi = __reduce_max_sync(0xffffffffu, hi);
    if ((ft & 31) == 0) ts.red[buf][ft >> 5] = hi;
    if (ft == 0) ts.n_trim = 0;
    fin_sync(team);
#pragma unroll
    for (int i = 0; i < kFinWarps; i++) hi = max(hi, ts.red[buf][i]);
    buf ^= 1;
    int left = n;
    while (lo < hi && left > k + 32 + k / 4) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      uint32_t c = 0;
      for (int i = ft; i < n; i += kFin) c += (uint32_t)(ts.cand[i] >> 32) >= mid;
      c = fin_sum(c, ts, team, buf);
      if ((int)c >= k) lo = mid, left = c;
      else hi = mid - 1;
    }
    for (int i = ft; i < n; i += kFin)
      if ((uint32_t)(ts.cand[i] >> 32) >= lo) {
        const int at = atomicAdd(&ts.n_trim, 1);
        if (at < kMaxTrim) ts.trim[at] = ts.cand[i];
      }
    fin_sync(team);
    if (ts.n_trim <= kMaxTrim) {
      n = ts.n_trim;
      from = ts.trim;
    }
  }
  for (int c = ft; c < n; c += 2 * kFin) {
    const bool two = c + kFin < n;
    const unsigned long long x = from[c], y = two ? from[c + kFin] : 0;
    int rx = 0, ry = 0;
#pragma unroll 8
    for (int i = 0; i < n; i++) {
      const unsigned long long o = from[i];
      rx += o > x;
      ry += o > y;
    }
    if (rx < k) ts.sorted[rx] = x;
    if (two && ry < k) ts.sorted[ry] = y;
  }
  fin_sync(team);
  return min(n, k);
}

// The k largest entries of a CTA's part of a row, best first, in ts.sorted; returns how many
// (fewer than k only where the part has no more that are not NaN).  Called by the finishers.
//
// The consumers leave the largest entry that each thread saw, and that of each bin of its
// vectors.  The k-th largest of the 512 threads' maxima, tau, is a lower bound of the part's
// k-th largest entry, so only bins that reach tau are read again (from L2): for entries in
// no order about 512 ln(512 / (512 - k)) bins, 21 for k = 20 and 147 for k = 128, of 16 to 32
// entries.  Every warp finds tau for itself, 16 maxima a lane, by a bisection over the keys
// that stops at a few threads more than k.  Arrives on `read` when the maxima are read, well
// before the end.
template <typename T>
__device__ int part_top(const T* row, const ScoreParams& p, TopSmem& ts, uint64_t* read, int team, int it, int v0,
                        int nvec, int tail_n, float tail_x) {
  using VT = Vec<T>;
  constexpr int E = VT::E, kKeys = kCons / 32;
  const int ft = fin_thread(team), lane = threadIdx.x & 31;
  const int k = p.k;
  const int n_st = (nvec + p.ring.stage - 1) / p.ring.stage, n_sub = p.ring.stage / kSub;
  const int per_bin = (p.subs + p.bins - 1) / p.bins;   // most turns of a bin
  if (ft == 0) ts.n_hits = ts.n_cand = 0;
  uint32_t lo, hi;
  bool exact = false;
  {
    uint32_t key[kKeys];
    uint32_t mn = 0xffffffffu, mx = 0;
#pragma unroll
    for (int i = 0; i < kKeys; i++) {
      key[i] = nvec > 0 ? order_key(ts.tmax[i * 32 + lane]) : order_key(-INFINITY);
      mn = min(mn, key[i]);
      mx = max(mx, key[i]);
    }
    lo = __reduce_min_sync(0xffffffffu, mn);
    hi = __reduce_max_sync(0xffffffffu, mx);
    auto count = [&](uint32_t t) {
      uint32_t c[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kKeys; i++) c[i & 3] += key[i] >= t;
      return __reduce_add_sync(0xffffffffu, (c[0] + c[1]) + (c[2] + c[3]));
    };
    // at least k threads (kCons >= kMaxTop) reach lo; fewer than k reach hi + 1
    if (lo <= order_key(-INFINITY) && (int)count(lo + 1) < k) hi = lo;
    const int enough = k + 8 + k / 4;
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      const int c = (int)count(mid);
      if (c >= k) {
        lo = mid;
        if (c <= enough) break;
      } else {
        hi = mid - 1;
      }
    }
    exact = lo == hi;
  }
  fin_sync(team);
  // bins that reach `from`
  auto find_bins = [&](uint32_t from) {
    const float ff = order_value(from);
    if (nvec > 0)
#pragma unroll
      for (int t = ft; t < kCons; t += kFin)
        if (ts.tmax[t] >= ff) {
          uint32_t hit = 0;
#pragma unroll
          for (int j = 0; j < kMaxBins; j++) hit |= (uint32_t)(j < p.bins && ts.bmax[j][t] >= ff) << j;
          int i = atomicAdd(&ts.n_hits, __popc(hit));
          for (; hit; hit &= hit - 1, i++)
            if (i < kMaxHits) ts.hit[i] = (uint16_t)((__ffs(hit) - 1) * kCons + t);
        }
    fin_sync(team);
    return ts.n_hits <= kMaxHits;
  };
  auto release = [&] {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(read);
  };
  // their entries of at least `from`, into cand
  auto collect = [&](uint32_t from) {
    const float ff = order_value(from);
    constexpr int U = 4;
    const int items = ts.n_hits * kPer * per_bin;
    for (int base = ft; base < items; base += U * kFin) {
      uint4 w[U];
      int at[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int item = base + u * kFin;
        at[u] = -1;
        if (item >= items) continue;
        const int h = per_bin == 1 ? item / kPer : item / (kPer * per_bin), q = item % kPer;
        const int bin = ts.hit[h] / kCons, t = ts.hit[h] % kCons, group = t / kGroupThreads;
        // the bin's turns: those with turn bins / subs = bin
        int turn = bin;
        if (p.subs > p.bins) {
          turn = (bin * p.subs + p.bins - 1) / p.bins + (item / kPer - h * per_bin);
          if (turn >= p.subs || turn * p.bins / p.subs != bin) continue;
        }
        const int j = first_stage(group, it, n_st) + turn / n_sub * kGroups;
        const int i = j * p.ring.stage + turn % n_sub * kSub + q * kGroupThreads + t % kGroupThreads;
        if (j >= n_st || i >= nvec) continue;
        at[u] = v0 + i;
        w[u] = reinterpret_cast<const uint4*>(row)[at[u]];
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        if (at[u] < 0) continue;
        float x[E];
        VT::cvt(w[u], x);
        uint32_t hit = 0;
#pragma unroll
        for (int e = 0; e < E; e++) hit |= (uint32_t)(x[e] >= ff) << e;
        if (!hit) continue;
        int c = atomicAdd(&ts.n_cand, __popc(hit));
#pragma unroll
        for (int e = 0; e < E; e++)
          if (hit >> e & 1) {
            if (c < kMaxCand) ts.cand[c] = cand_of(order_key(x[e]), at[u] * E + e);
            c++;
          }
      }
      if (ts.n_cand > kMaxCand) break;   // too many: all of it is done again
    }
    if (ft < tail_n && tail_x >= ff) {
      const int c = atomicAdd(&ts.n_cand, 1);
      if (c < kMaxCand) ts.cand[c] = cand_of(order_key(tail_x), p.V - tail_n + ft);
    }
    fin_sync(team);
    return ts.n_cand <= kMaxCand;
  };
  int buf = 0;
  auto reset = [&] {
    fin_sync(team);
    if (ft == 0) ts.n_hits = ts.n_cand = ts.n_ties = 0;
    fin_sync(team);
  };
  bool slow;
  if (lo > order_key(-INFINITY) && find_bins(lo)) {
    release();
    if (collect(lo)) return rank_cand(ts, team, k, lo, buf);
    slow = true;
  } else {
    // Most bins reach tau, as with equal entries in all of them (masked rows, rounded
    // logits).  With the exact tau fewer than k threads exceed it: take what exceeds tau, and
    // the entries equal to it in the order of their ids.
    while (!exact && lo < hi) {
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      uint32_t c = 0;
      for (int i = 0; i < kKeys; i++) c += nvec > 0 && order_key(ts.tmax[i * 32 + lane]) >= mid;
      c = __reduce_add_sync(0xffffffffu, c);
      if ((int)c >= k) lo = mid;
      else hi = mid - 1;
    }
    reset();
    slow = !find_bins(lo + 1);
    release();
    slow = slow || !collect(lo + 1);
  }
  if (slow) {
    // Few bins hold more than kMaxCand entries that reach tau: find the part's k-th largest
    // entry by counting over the whole part, up to 32 times.  Slow, for rows whose k-th largest
    // value is shared by thousands of neighbouring entries: rows of 151,936 bf16 masked but for
    // 2,000 adjacent equal ones take 317 us (one row) and 1.3 ms (256 rows) with their top 20,
    // random rows 13 and 22 us.  1,200 such entries, ranked as candidates, take 70 and 105 us.
    uint32_t a = lo, b = 0xffffffffu;
    while (a < b) {
      const uint32_t mid = a + (b - a) / 2 + ((b - a) & 1);
      uint32_t c = ft < tail_n && order_key(tail_x) >= mid;
      for (int i = ft; i < nvec; i += kFin) {
        float x[E];
        VT::cvt(*reinterpret_cast<const uint4*>(row + (size_t)(v0 + i) * E), x);
#pragma unroll
        for (int e = 0; e < E; e++) c += order_key(x[e]) >= mid;
      }
      c = fin_sum(c, ts, team, buf);
      if ((int)c >= k) a = mid;
      else b = mid - 1;
    }
    lo = a;   // fewer than k entries exceed it
    reset();
    for (int i = ft; i < nvec; i += kFin) {
      float x[E];
      VT::cvt(*reinterpret_cast<const uint4*>(row + (size_t)(v0 + i) * E), x);
#pragma unroll
      for (int e = 0; e < E; e++) {
        const uint32_t kx = order_key(x[e]);
        if (kx > lo) ts.cand[atomicAdd(&ts.n_cand, 1)] = cand_of(kx, (v0 + i) * E + e);
      }
    }
    if (ft < tail_n && order_key(tail_x) > lo)
      ts.cand[atomicAdd(&ts.n_cand, 1)] = cand_of(order_key(tail_x), p.V - tail_n + ft);
    fin_sync(team);
  }
  const int above = ts.n_cand;
  // ties by id: 128 vectors at a time, then the last entries, until there are enough
  int found = 0;
  for (int base = 0; base < nvec + 1 && above + found < k; base += kFin) {
    uint32_t hit = 0;
    const int i = base + ft;
    if (i < nvec) {
      float x[E];
      VT::cvt(*reinterpret_cast<const uint4*>(row + (size_t)(v0 + i) * E), x);
#pragma unroll
      for (int e = 0; e < E; e++) hit |= (uint32_t)(order_key(x[e]) == lo) << e;
    }
    const int mine = __popc(hit);
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) ts.red[buf][ft >> 5] = inc;
    fin_sync(team);
    int at = found + inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kFinWarps; w++) {
      if (w < (ft >> 5)) at += ts.red[buf][w];
      total += ts.red[buf][w];
    }
    buf ^= 1;
    for (int e = 0; e < E; e++)
      if (hit >> e & 1) {
        if (above + at < k) ts.cand[above + at] = cand_of(lo, (v0 + i) * E + e);
        at++;
      }
    found += total;
  }
  if (ft < 32) {
    const bool hit = ft < tail_n && order_key(tail_x) == lo;
    const uint32_t who = __ballot_sync(0xffffffffu, hit);
    const int at = above + found + __popc(who & ((1u << lane) - 1));
    if (hit && at < k) ts.cand[at] = cand_of(lo, p.V - tail_n + ft);
    if (ft == 0) ts.n_ties = found + __popc(who);
  }
  fin_sync(team);
  if (above < k) {
    if (ft == 0) ts.n_cand = min(above + ts.n_ties, k);
    fin_sync(team);
  }
  return rank_cand(ts, team, k, lo, buf);
}

// Of a masked entry -inf, also where all of the row are (ls = -inf), but NaN in a row of a NaN or
// +inf logit (ls NaN).
__device__ __forceinline__ float log_prob(float x, float m, float ls, float c) {
  return x == -INFINITY && ls == ls ? -INFINITY : (x - m) * c - ls;
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kBlock, 1) k_token_score(const __grid_constant__ ScoreParams p) {
  using VT = Vec<T>;
  constexpr int E = VT::E;
  extern __shared__ __align__(128) uint8_t smem[];
  ScoreSmem& ss = *reinterpret_cast<ScoreSmem*>(smem);
  TopSmem* const top = reinterpret_cast<TopSmem*>(smem + (sizeof(ScoreSmem) + 15) / 16 * 16);
  uint4* const slots = reinterpret_cast<uint4*>(smem + ring_offset<kTop>());
  RingBars& bar = ss.bars;
  const RingShape rs = p.ring;
  const uint32_t rank = rs.cs > 1 ? cluster_rank() : 0;
  const int n_clusters = gridDim.x / rs.cs, cluster = blockIdx.x / rs.cs;
  const int nv = p.V / E;
  const int v0 = min(nv, (int)rank * rs.seg), nvec = min(rs.seg, nv - v0);
  const int tid = threadIdx.x, lane = tid & 31;
  const float c2 = p.c * kLog2e;
  const T* const logits = reinterpret_cast<const T*>(p.logits);

  if (tid == 0) bar.init(kFinWarps);
  __syncthreads();
  if (rs.cs > 1) cluster_sync();
  wait_for_predecessor();

  if (tid >= kLook && tid < kFirstCons) {
    // ---- look-ups: the tokens that the rows feed, 32 rows at a time, a lane for each ----
    if (rank == 0 && p.ids) {
      auto token = [&](const T* row, int t, float* x) {   // whether its id is one
        const int id = p.ids[t];
        const bool good = id >= 0 && id < p.V;
        if (good) *x = VT::get(row + id);
        else atomicExch(p.status, OCTO_EINVAL);
        return good;
      };
      bool ok = true;
      for (int first = 0; ok && cluster + first * n_clusters < p.n; first += 32) {
        const int mine = cluster + (first + lane) * n_clusters, r = p.row0 + mine;
        int t = -1, e0 = 0, n = 0;
        float x = 0.f;
        bool good = false;
        if (mine < p.n) {
          if (p.succ.is_decode) {
            t = r;
          } else {
            int end;
            bool start;
            p.succ.locate(r, &end, &start, &e0, &n);
            if (r + 1 < end) t = r + 1;
            if (start) p.logp[r] = 0.f;
          }
          if (t >= 0) good = token(logits + (size_t)mine * p.ld, t, &x);
        }
        for (int j = 0; j < 32; j++) {
          const int it = first + j, rl = cluster + it * n_clusters, par = it & 1;
          if (rl >= p.n) break;
          if (!(ok = warp_wait(&bar.scal_full[par], (it >> 1) & 1, p.status))) break;
          const float m = ss.stat[par][0], ls = ss.stat[par][1];
          if (lane == j && t >= 0) p.logp[t] = good ? log_prob(x, m, ls, p.c) : __int_as_float(0x7fc00000);
          const int more = __shfl_sync(0xffffffffu, n, j), at = __shfl_sync(0xffffffffu, e0, j);
          for (int i = lane; i < more; i += 32) {   // a fork's or a rewind's
            const int t2 = p.succ.ex_row[at + i];
            float x2 = 0.f;
            const bool good2 = token(logits + (size_t)rl * p.ld, t2, &x2);
            p.logp[t2] = good2 ? log_prob(x2, m, ls, p.c) : __int_as_float(0x7fc00000);
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bar.scal_empty[par]);   // after what used them
        }
      }
    }
  } else if (tid >= kCopy && tid < kLook) {
    // ---- copies ----
    if (lane == 0) {
      RingPos pos;
      int issued = 0;
      bool ok = true;
      for (int r = cluster; r < p.n && ok; r += n_clusters) {
        const T* src = logits + (size_t)r * p.ld + (size_t)v0 * E;
        for (int b = 0; b < nvec; b += rs.stage) {
          if (!(ok = ring_wait(&bar.empty[pos.slot], pos.round ^ 1, p.status))) break;
          const uint32_t bytes = (uint32_t)min(rs.stage, nvec - b) * 16;
          tc::mbar_expect_tx(&bar.full[pos.slot], bytes);
          bulk_load(slots + (size_t)pos.slot * rs.stage, src + (size_t)b * E, bytes, &bar.full[pos.slot]);
          pos.skip(1, rs.n_slots);
          issued++;
        }
      }
      // a copy must not outlive the CTA: the consumers have seen all of them unless a wait gave up
      if (!ok)
        for (int i = min(issued, rs.n_slots); i > 0; i--) {
          if (--pos.slot < 0) pos.slot = rs.n_slots - 1, pos.round ^= 1;
          ring_wait(&bar.full[pos.slot], pos.round, p.status);
        }
    }
  } else if (tid >= kFirstCons) {
    // ---- consumers: sums of the part, maxima of the bins ----
    const int ct = tid - kFirstCons, group = ct / kGroupThreads, t = ct % kGroupThreads;
    const int n_st = (nvec + rs.stage - 1) / rs.stage, n_sub = rs.stage / kSub;
    RingPos pos;
    pos.skip(group, rs.n_slots);
    bool ok = true;
    StageStat<T, true> st;
    for (int r = cluster, it = 0; r < p.n && ok; r += n_clusters, it++) {
      const int par = it & 1;
      st.init();
      float bm = -INFINITY, tm = -INFINITY;
      int bin = 0, frac = 0;
      // the finishers are done with this parity's buffers two rows ago
      if (kTop) ok = warp_wait(&bar.part_empty[par], ((it >> 1) & 1) ^ 1, p.status);
      for (int j = first_stage(group, it, n_st); j < n_st && ok; j += kGroups) {
        if (!(ok = warp_wait(&bar.full[pos.slot], pos.round, p.status))) break;
        const uint4* slot = slots + (size_t)pos.slot * rs.stage;
        const int cnt = nvec - j * rs.stage;
        for (int u = 0; u < n_sub; u++) {
          const int left = cnt - u * kSub;
          if (left > 0) {
            uint4 w[kPer];
            load_sub<T>(slot + u * kSub, left, t, w);
            const float mx = Raw<T>::max(w);
            if (u + 1 == n_sub || left <= kSub) give_back(&bar.empty[pos.slot], mx);
            tm = fmaxf(tm, mx);
            bm = fmaxf(bm, mx);
            st.add(w, left, mx, c2);
          }
          if (kTop && (frac += p.bins) >= p.subs) {
            frac -= p.subs;
            top[par].bmax[bin++][ct] = bm;
            bm = -INFINITY;
          }
        }
        pos.skip(kGroups, rs.n_slots);
      }
      if (!ok) break;
      if (kTop) {
        for (; bin < p.bins; bin++) top[par].bmax[bin][ct] = bm, bm = -INFINITY;
        top[par].tmax[ct] = tm;
      }
      Stat tot = st.total(tm, c2);
      warp_merge(tot, c2);
      if (!kTop) ok = warp_wait(&bar.part_empty[par], ((it >> 1) & 1) ^ 1, p.status);
      if (lane == 0) {
        float* q = ss.part[par][ct >> 5];
        q[0] = tot.m, q[1] = tot.s, q[2] = tot.a;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar.part_full[par]);
    }
  } else {
    // ---- finishers: team `par` takes the rows of that parity ----
    const int par = tid / kFin, ft = fin_thread(par);
    TopSmem& ts = top[par];
    const int tail_n = rank + 1 == (uint32_t)rs.cs ? p.V - nv * E : 0;
    for (int r = cluster + par * n_clusters, it = par; r < p.n; r += 2 * n_clusters, it += 2) {
      const uint32_t ph = (it >> 1) & 1;
      const T* row = logits + (size_t)r * p.ld;
      const float tail_x = ft < tail_n ? VT::get(row + nv * E + ft) : -INFINITY;
      if (!fin_all(ring_wait(&bar.part_full[par], ph, p.status), par)) break;
      Stat st;
      st.init();
      if (lane < kConsWarps) {
        const float* q = ss.part[par][lane];
        st.m = q[0], st.s = q[1], st.a = q[2];
      } else if (lane - kConsWarps < tail_n) {
        const float x = VT::get(row + nv * E + lane - kConsWarps);
        if (x > st.m) st.m = x;
        st.add(x, c2);
      }
      warp_merge(st, c2);
      int n_top = 0;
      if (kTop) {
        n_top = part_top<T>(row, p, ts, &bar.part_empty[par], par, it, v0, nvec, tail_n, tail_x);
      } else {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bar.part_empty[par]);
      }

      if (rs.cs > 1) {
        // to rank 0 (a cluster of several CTAs has a single row: nothing is sent twice)
        uint64_t* const joined = &bar.joined[par][0];
        const uint32_t far = map_rank(tc::smem_u32(joined), 0);
        if (rank == 0 && ft == 0) tc::mbar_expect_tx(joined, rs.cs * (16 + 8 * p.k));
        if (kTop && ft < p.k)   // places that are left over are 0
          st_async(map_rank(tc::smem_u32(&ts.in_list[rank][ft]), 0), ft < n_top ? ts.sorted[ft] : 0ull, far);
        if (ft == 0) st_async(map_rank(tc::smem_u32(ss.in_stat[rank]), 0), st.m, st.s, st.a, 0.f, far);
        if (rank != 0) continue;
        if (!fin_all(ring_wait<true>(joined, ph, p.status), par)) break;
        uint32_t bound = 1;   // the k-th best of any full list is a lower bound of the row's
        st.init();
        for (int q = 0; q < rs.cs; q++) st.merge(ss.in_stat[q][0], ss.in_stat[q][1], ss.in_stat[q][2], c2);
        if (kTop) {
          for (int q = 0; q < rs.cs; q++) {
            if (ft < p.k) ts.cand[q * p.k + ft] = ts.in_list[q][ft];
            bound = max(bound, (uint32_t)(ts.in_list[q][p.k - 1] >> 32));
          }
          if (ft < p.k) ts.sorted[ft] = 0;
          if (ft == 0) ts.n_cand = rs.cs * p.k;
        }
        fin_sync(par);
        int buf = 0;
        if (kTop) n_top = rank_cand(ts, par, p.k, bound, buf);
      }
      const bool empty = st.s == 0.f;
      const float m = empty ? -INFINITY : st.m, ls = empty ? -INFINITY : logf(st.s);
      if (ft == 0) {
        p.row_stat[2 * (size_t)r] = m;
        p.row_stat[2 * (size_t)r + 1] = ls;
        if (p.entropy) p.entropy[r] = empty ? 0.f : ls - kLn2 * (st.a / st.s);
        if (p.ids) {
          ring_wait(&bar.scal_empty[par], ph ^ 1, p.status);
          ss.stat[par][0] = m;
          ss.stat[par][1] = ls;
          tc::mbar_arrive(&bar.scal_full[par]);
        }
      }
      if (kTop && ft < p.k) {
        const unsigned long long e = ft < n_top ? ts.sorted[ft] : 0;
        const size_t o = (size_t)r * p.k + ft;
        p.top_ids[o] = e ? (int32_t) ~(uint32_t)e : -1;
        p.top_logp[o] = e ? log_prob(order_value((uint32_t)(e >> 32)), m, ls, p.c) : __int_as_float(0x7fc00000);
      }
    }
  }
  // no CTA leaves while another may still write to its shared memory
  __syncwarp();
  if (rs.cs > 1) cluster_sync();
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
  int32_t parts, part_vecs;   // CTAs per row, vectors of each
};

// In log2 units, y = c2 (x - m) - log2 S and p = 2^y, an element's gradient is p (A + B y)
// with the row's A = -c (G + g_H H), B = -c g_H ln 2, plus c g_t at the successors' ids.
//
// One pass, bound by memory: a CTA takes up to kThreads * kBwdPer vectors of a row, all of its
// loads in flight before it looks up the row's successors.  6,144 rows of 151,936 bf16, with
// 2 / 3 / 4 / 6 / 8 vectors a thread and as many CTAs as their registers leave: 698 / 567 /
// 542 / 554 / 570 us (6.9 TB/s).
constexpr int kBwdPer = 4;

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, 1536 / kThreads) k_token_score_bwd(const __grid_constant__ ScoreBwdParams p) {
  using VT = Vec<T>;
  constexpr int E = VT::E;
  __shared__ int32_t s_t[kMaxSucc], s_id[kMaxSucc];
  __shared__ float s_g[kMaxSucc];
  __shared__ float s_G;
  __shared__ int32_t s_n, s_lo, s_hi;
  const int rl = blockIdx.x / p.parts, part = blockIdx.x - rl * p.parts, tid = threadIdx.x;
  const T* row = reinterpret_cast<const T*>(p.logits) + (size_t)rl * p.ld;
  T* grow = reinterpret_cast<T*>(p.dlogits) + (size_t)rl * p.ld;
  const int nv = p.V / E, v0 = part * p.part_vecs, v1 = min(nv, v0 + p.part_vecs);
  wait_for_predecessor();
  uint4 w[kBwdPer];
#pragma unroll
  for (int q = 0; q < kBwdPer; q++) {
    const int i = v0 + q * kThreads + tid;
    if (i < v1) w[q] = __ldcs(reinterpret_cast<const uint4*>(row) + i);
  }
  const float m = p.row_stat[2 * (size_t)rl], ls = p.row_stat[2 * (size_t)rl + 1];
  const float gH = p.g_entropy ? p.g_entropy[rl] : 0.f, H = p.g_entropy ? p.entropy[rl] : 0.f;
  if (tid < 32) {
    int nt = 0;
    if (p.g_logp) {
      nt = p.succ.find(p.row0 + rl, s_t);
      __syncwarp();
      for (int i = tid; i < nt; i += 32) {
        const int t = s_t[i], id = p.ids[t];
        const bool bad = id < 0 || id >= p.V;
        if (bad) atomicExch(p.status, OCTO_EINVAL);
        s_id[i] = bad ? -1 : id;
        s_g[i] = bad ? 0.f : p.g_logp[t];
      }
      __syncwarp();
    }
    if (tid == 0) {
      float G = 0.f;
      int lo = p.V, hi = -1;
      for (int i = 0; i < nt; i++) {
        if (s_id[i] < 0) continue;
        G += s_g[i];
        lo = min(lo, s_id[i]);
        hi = max(hi, s_id[i]);
      }
      s_n = nt, s_G = G, s_lo = lo, s_hi = hi;
    }
  }
  __syncthreads();
  const int lo = s_lo, hi = s_hi;
  const float A = -p.c * (s_G + gH * H), B = -p.c * kLn2 * gH;
  auto onehot = [&](int v) {
    float g = 0.f;
    for (int i = 0; i < s_n; i++)
      if (s_id[i] == v) g += s_g[i];
    return p.c * g;
  };
  if (m == -INFINITY) {   // nothing left in the row
    for (int i = v0 + tid; i < v1; i += kThreads) __stcs(reinterpret_cast<uint4*>(grow) + i, make_uint4(0, 0, 0, 0));
    if (v1 == nv && tid < p.V - nv * E) VT::put(grow + nv * E + tid, 0.f);
    return;
  }
  const float c2 = p.c * kLog2e, l2 = ls * kLog2e;
  const f2 negm = pack2(-m, -m), cc = pack2(c2, c2), nl = pack2(-l2, -l2), AA = pack2(A, A), BB = pack2(B, B);
#pragma unroll
  for (int q = 0; q < kBwdPer; q++) {
    const int i = v0 + q * kThreads + tid;
    if (i < v1) {
      float g[E];
#pragma unroll
      for (int e = 0; e < E / 2; e++) {
        float y0, y1;
        unpack2(fma2(add2(Raw<T>::pair(w[q], e), negm), cc, nl), y0, y1);
        y0 = max_nan(y0, kCut);
        y1 = max_nan(y1, kCut);
        unpack2(mul2(pack2(ex2f(y0), ex2f(y1)), fma2(BB, pack2(y0, y1), AA)), g[2 * e], g[2 * e + 1]);
      }
      if (i * E <= hi && i * E + E - 1 >= lo) {
#pragma unroll
        for (int e = 0; e < E; e++) g[e] += onehot(i * E + e);
      }
      __stcs(reinterpret_cast<uint4*>(grow) + i, VT::pack(g));
    }
  }
  if (v1 == nv && tid < p.V - nv * E) {
    const int v = nv * E + tid;
    const float y = max_nan((VT::get(row + v) - m) * c2 - l2, kCut);
    VT::put(grow + v, ex2f(y) * fmaf(B, y, A) + onehot(v));
  }
}

template <typename T, bool kTop>
int launch_score(ScoreParams& p, cudaStream_t s) {
  const int off = ring_offset<kTop>(), ring = kSmemMax - off;
  const int64_t nv = p.V / Vec<T>::E;
  const void* f = (const void*)k_token_score<T, kTop>;
  int cs = 1;
  // measured at 32,000 and 151,936 entries, one row: joining 2 to 8 sums takes 0.5 to 0.9 us,
  // joining their alternatives 1.4 us at k = 20 and 2 CTAs, 2.5 at 8, and up to 2 more at k = 128
  // (one row of 151,936 in bf16, 1 / 2 / 4 / 8 CTAs: 9.3 / 7.4 / 6.3 / 5.6 us at k = 0,
  // 13.4 / 12.5 / 11.8 / 11.8 at k = 20)
  const int k = p.k;
  if (int st = pick_cluster(f, p.n, nv, kSmemMax, [k](int c) { return k ? 1.2 + 0.015 * k + 0.15 * c : 0.7; }, &cs)) return st;
  p.ring = ring_shape(nv, cs, ring);
  p.subs = std::max(1, (p.ring.n_stages + kGroups - 1) / kGroups * (p.ring.stage / kSub));
  p.bins = std::min(p.subs, kMaxBins);
  return launch_ring(f, p, p.n, cs, off + p.ring.n_slots * p.ring.stage * 16, s);
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
  p.n = n_rows;
  const bool bf = dtype == OCTO_DTYPE_BF16;
  if (k > 0) return bf ? launch_score<__nv_bfloat16, true>(p, s) : launch_score<float, true>(p, s);
  return bf ? launch_score<__nv_bfloat16, false>(p, s) : launch_score<float, false>(p, s);
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
  const bool bf = dtype == OCTO_DTYPE_BF16;
  const int32_t vecs = vocab / (bf ? 8 : 4);
  // Short rows: a CTA is mostly waiting for its look-ups, so many small ones (1,360 rows of
  // 256 / 1,500 entries: 11 -> 5 / 12 -> 10 us); with few rows 256 threads are no slower.
  const int threads = vecs <= 64 * kBwdPer && n_rows > 4 * sm_count() ? 64 : 256, most = threads * kBwdPer;
  p.parts = vecs > most ? (vecs + most - 1) / most : 1;
  p.part_vecs = (vecs + p.parts - 1) / p.parts;
  if ((int64_t)n_rows * p.parts > INT32_MAX) return OCTO_EINVAL;
  const int grid = n_rows * p.parts;
  const void* f = threads == 64 ? (bf ? (const void*)k_token_score_bwd<__nv_bfloat16, 64> : (const void*)k_token_score_bwd<float, 64>)
                                : (bf ? (const void*)k_token_score_bwd<__nv_bfloat16, 256> : (const void*)k_token_score_bwd<float, 256>);
  return launch_overlapped(f, &p, grid, threads, 1, 0, s);
}

}  // extern "C"
