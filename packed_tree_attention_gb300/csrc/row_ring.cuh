// Rows of logits streamed through a ring of shared-memory slots: the frame of the token
// scoring and distillation kernels.
//
// A cluster of `cs` CTAs takes one row after another; each CTA has its own contiguous part of
// the row's 16-byte vectors.  One thread copies the part, stage by stage, into the ring with
// bulk copies (cp.async.bulk, completion on a slot's `full` barrier), running ahead over row
// ends as far as the ring reaches; four groups of 4 consumer warps take the stages in turn, so
// that the waits of one fall into the arithmetic of another; 8 finisher warps, in teams that
// take the rows in turn, do what a row needs besides, while the consumers are at the next ones.
// One CTA per SM, the grid as many clusters as the device holds.
// The copies bring whole vectors: the last V % E entries are the finishers'.
#pragma once

#include "row_common.cuh"
#include "tc_common.cuh"

namespace octo {
namespace rows {

constexpr int kConsWarps = 16, kCons = kConsWarps * 32;
constexpr int kFinishers = 8;               // warps; teams of 4 (scoring) or of 1 (distillation)
// Warps: the finishers, the copying one, one for look-ups, the consumers.
constexpr int kCopy = kFinishers * 32, kLook = kCopy + 32, kFirstCons = kLook + 32;
constexpr int kBlock = kFirstCons + kCons;
constexpr int kGroups = 4;                  // consumer groups, a warp of each on every scheduler
constexpr int kGroupThreads = kCons / kGroups;
constexpr int kPer = 4;                     // vectors that a thread takes at once
constexpr int kSub = kPer * kGroupThreads;  // and a group: stages are multiples of that
constexpr int kMaxSlots = 28;
constexpr int kMaxCluster = 8;
constexpr int kMaxRows = kFinishers;        // rows that a CTA works on at once

struct RingShape {
  int32_t cs;          // CTAs per row
  int32_t seg;         // vectors of a CTA's part (the last ones may have fewer)
  int32_t stage;       // vectors of a slot
  int32_t n_stages;    // stages of a part
  int32_t n_slots;
};

// cs CTAs per row, ring of at most `bytes`, stages of 1, 2 or 4 kSub.  Short stages give every
// group its share of a short part, long ones cost fewer waits.  The slots are a multiple of the
// groups, so that a slot is always the same group's: copies complete in no order, and a parity
// wait on a slot whose last stage, another group's, had not come would take that phase's
// predecessor for its own.
inline RingShape ring_shape(int64_t nv, int cs, int bytes) {
  RingShape s;
  s.cs = cs;
  s.seg = (int32_t)((nv + cs - 1) / cs);
  s.stage = kSub * (s.seg <= 8 * kSub ? 1 : s.seg <= 40 * kSub ? 2 : 4);
  s.n_stages = (s.seg + s.stage - 1) / s.stage;
  s.n_slots = bytes / (s.stage * 16);
  if (s.n_slots > kMaxSlots) s.n_slots = kMaxSlots;
  s.n_slots -= s.n_slots % kGroups;
  return s;
}

// last: nothing reads the bytes again, L2 may drop them first.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, bool last = false) {
  if (last) {
    uint64_t policy;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                     tc::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar)), "l"(policy)
                 : "memory");
    return;
  }
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   tc::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
               : "memory");
}

// Waits of these kernels: a poll suspends the thread for up to kPollNs (it wakes when the phase
// completes), so that waiting warps leave the issue slots to the others; given up after
// kPolls of them, several seconds.
constexpr uint32_t kPollNs = 1000000, kPolls = 4000;
template <bool kCluster = false>
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  const uint32_t a = tc::smem_u32(bar);
#pragma unroll 1
  for (uint32_t i = 0; i < kPolls; i++) {
    uint32_t ok;
    if (kCluster)   // what the peers stored before they arrived is visible after it
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(a), "r"(parity), "r"(kPollNs)
          : "memory");
    else
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(ok)
          : "r"(a), "r"(parity), "r"(kPollNs)
          : "memory");
    if (ok) return true;
  }
  atomicExch(status, OCTO_ETIMEOUT);
  return false;
}
// Uniform over the warp: after a wait that gave up, its lanes leave together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, ring_wait(bar, parity, status));
}

// Launched so that its start overlaps the end of the kernel before it, a kernel waits here before
// it touches global memory.
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the kernel after it, if that waits so, be launched once every CTA has come here.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- clusters ----
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
// Stores to a peer's shared memory that count their bytes on a barrier of the peer's.  (An
// arrival with release semantics would wait for the thread's earlier global stores first.)
__device__ __forceinline__ void st_async(uint32_t a, float x, float y, float z, float w, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a), "f"(x),
               "f"(y), "f"(z), "f"(w), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void st_async(uint32_t a, unsigned long long v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(a), "l"(v), "r"(bar) : "memory");
}

// ---- two fp32 operations per instruction ----
typedef unsigned long long f2;
__device__ __forceinline__ f2 pack2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  static constexpr int kPairs = 4;
  __device__ __forceinline__ static uint4 masked() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
  __device__ __forceinline__ static f2 pair(const uint4& w, int i) {
    const uint32_t u = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return pack2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  // largest entry, NaNs left out, or NaN where one of them is (kNan)
  template <bool kNan = false>
  __device__ __forceinline__ static float max(const uint4 (&w)[kPer]) {
    auto b = [](uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); };
    auto of = [](__nv_bfloat162 x, __nv_bfloat162 y) { return kNan ? __hmax2_nan(x, y) : __hmax2(x, y); };
    auto h = [&](const uint4& v) { return of(of(b(v.x), b(v.y)), of(b(v.z), b(v.w))); };
    __nv_bfloat162 m = h(w[0]);
#pragma unroll
    for (int q = 1; q < kPer; q++) m = of(m, h(w[q]));
    return kNan ? max_nan(__low2float(m), __high2float(m)) : fmaxf(__low2float(m), __high2float(m));
  }
  // entries below -2^100 raised to it, NaNs kept
  __device__ __forceinline__ static uint4 floored(const uint4& w) {
    auto f = [](uint32_t u) {
      uint32_t r;
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0xf180f180u));
      return r;
    };
    return make_uint4(f(w.x), f(w.y), f(w.z), f(w.w));
  }
};
template <>
struct Raw<float> {
  static constexpr int kPairs = 2;
  __device__ __forceinline__ static uint4 masked() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
  __device__ __forceinline__ static f2 pair(const uint4& w, int i) {
    return i == 0 ? pack2(__uint_as_float(w.x), __uint_as_float(w.y)) : pack2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  template <bool kNan = false>
  __device__ __forceinline__ static float max(const uint4 (&w)[kPer]) {
    auto of = [](float x, float y) { return kNan ? max_nan(x, y) : fmaxf(x, y); };
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < kPer; q++)
      m = of(m, of(of(__uint_as_float(w[q].x), __uint_as_float(w[q].y)), of(__uint_as_float(w[q].z), __uint_as_float(w[q].w))));
    return m;
  }
  __device__ __forceinline__ static uint4 floored(const uint4& w) {
    auto f = [](uint32_t u) { return __float_as_uint(max_nan(__uint_as_float(u), -0x1p100f)); };
    return make_uint4(f(w.x), f(w.y), f(w.z), f(w.w));
  }
};

// A thread's running statistics over stages, sums in pairs, two chains.  The reference m follows
// the largest entry only when that is more than 2^kSlack times as likely (with one stage's
// largest entry as the start, hardly ever): moving it costs as much as several entries, and a
// warp pays when one lane does.  total() refers the sums to the largest entry; the entropy's
// sum loses 2^-24 kSlack there at most.
//
// With a usual reference, of size below 2^96, the exponent of an entry is one fused
// multiply-add, t = c2 x - r with r = c2 m rounded: relative to r the sums are exact to the
// exponential's own error, and total() corrects by the rounding error of r, which an fma gives
// exactly.  Entries below -2^100 add nothing there and are raised to it, so that a masked one's
// term of the entropy is 0 and not 0 * inf.  Other references (below -2^96: nothing but masked
// entries so far), and temperatures that take c2 2^100 out of range, take the difference first
// and cut each exponent off.
constexpr float kSlack = 8.f;
template <typename T, bool kEntropy>
struct StageStat {
  float m, r;
  f2 s[2], a[2];
  __device__ __forceinline__ void init() { m = -FLT_MAX, r = 0.f, s[0] = s[1] = a[0] = a[1] = 0ull; }
  __device__ __forceinline__ static bool usual(float m, float c2) {
    return fabsf(m) < 0x1p96f && c2 < 0x1p20f && c2 > 0x1p-80f;
  }
  __device__ __forceinline__ void raise(float mn, float c2) {
    // r is the rounded product: the difference of two of them, the new one not fused into it
    const float rn = __fmul_rn(mn, c2);
    const float d = max_nan(usual(m, c2) ? __fsub_rn(r, rn) : (m - mn) * c2, kCut);
    const float e = ex2f(d);
    const f2 f = pack2(e, e), dd = pack2(d, d);
#pragma unroll
    for (int i = 0; i < 2; i++) {
      if (kEntropy) a[i] = mul2(f, fma2(dd, s[i], a[i]));
      s[i] = mul2(f, s[i]);
    }
    m = mn;
    r = rn;
  }
  template <bool kUsual>
  __device__ __forceinline__ void add_vec(const uint4& raw, float c2) {
    const uint4 w = kEntropy && kUsual ? Raw<T>::floored(raw) : raw;
    const f2 cc = pack2(c2, c2), neg = kUsual ? pack2(-r, -r) : pack2(-m, -m);
#pragma unroll
    for (int i = 0; i < Raw<T>::kPairs; i++) {
      f2 t = Raw<T>::pair(w, i);
      t = kUsual ? fma2(t, cc, neg) : mul2(add2(t, neg), cc);
      float t0, t1;
      unpack2(t, t0, t1);
      if (!kUsual) t0 = max_nan(t0, kCut), t1 = max_nan(t1, kCut), t = pack2(t0, t1);
      const f2 e = pack2(ex2f(t0), ex2f(t1));
      s[i & 1] = add2(s[i & 1], e);
      if (kEntropy) a[i & 1] = fma2(e, t, a[i & 1]);
    }
  }
  template <bool kUsual>
  __device__ __forceinline__ void add_all(const uint4 (&w)[kPer], int cnt, float c2) {
    if (cnt > (kPer - 1) * kGroupThreads) {
#pragma unroll
      for (int q = 0; q < kPer; q++) add_vec<kUsual>(w[q], c2);
    } else {
#pragma unroll
      for (int q = 0; q < kPer - 1; q++)
        if (q * kGroupThreads < cnt) add_vec<kUsual>(w[q], c2);
    }
  }
  // the vectors w[q] with q * kGroupThreads < cnt, the largest entry of all kPer being mx
  __device__ __forceinline__ void add(const uint4 (&w)[kPer], int cnt, float mx, float c2) {
    if ((mx - m) * c2 > kSlack) raise(mx, c2);
    if (usual(m, c2)) add_all<true>(w, cnt, c2);
    else add_all<false>(w, cnt, c2);
  }
  // statistics relative to the largest entry mx
  __device__ __forceinline__ Stat total(float mx, float c2) const {
    float x, y, z, w;
    unpack2(add2(s[0], s[1]), x, y);
    unpack2(add2(a[0], a[1]), z, w);
    Stat t{m, x + y, kEntropy ? z + w : 0.f};
    if (usual(m, c2)) {
      const float d = fmaf(-m, c2, r), f = ex2f(d);
      t.a = f * fmaf(d, t.s, t.a);
      t.s *= f;
    }
    if (mx > m) t.rebase(mx, c2);
    return t;
  }
};

// Merges the lanes' statistics, every lane gets the warp's: the common reference first, so
// that each lane moves to it once and the sums are plain additions, in a fixed order.
__device__ __forceinline__ void warp_merge(Stat& st, float c2) {
  float mn;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(mn) : "f"(st.m));
  st.rebase(mn, c2);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
    st.a += __shfl_xor_sync(0xffffffffu, st.a, o);
  }
}

// Thread t of a group: its kPer vectors of the cnt ones from `slot` on (masked past the end).
template <typename T>
__device__ __forceinline__ void load_sub(const uint4* slot, int cnt, int t, uint4 (&w)[kPer]) {
  if (cnt >= kSub) {
#pragma unroll
    for (int q = 0; q < kPer; q++) w[q] = slot[q * kGroupThreads + t];
  } else {
#pragma unroll
    for (int q = 0; q < kPer; q++) {
      const int i = q * kGroupThreads + t;
      w[q] = i < cnt ? slot[i] : Raw<T>::masked();
    }
  }
}

// Gives a slot back once the warp's loads of it have returned, mx being a value made of them.
// An arrival right after the loads overtakes them: they queue behind other warps' misses
// (scattered loads at a kernel's start take microseconds), and the next copy came into the slot
// before they were served, 128 bytes here and there.  So the arrival is made to need mx: both
// of its forms do the same.
__device__ __forceinline__ void give_back(uint64_t* empty, float mx) {
  const uint32_t v = __ballot_sync(0xffffffffu, __float_as_uint(mx) != 0x7fedcba9u);
  if ((threadIdx.x & 31) == 0)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t"
        "@!p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(tc::smem_u32(empty)),
        "r"(v)
        : "memory");
}

// The barriers of a CTA; those of a row by its turn among the rows in work.
struct RingBars {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t part_full[kMaxRows], part_empty[kMaxRows];   // warp sums: written, read
  uint64_t joined[kMaxRows][2];                         // the bytes that the cluster's CTAs send
  uint64_t scal_full[kMaxRows], scal_empty[kMaxRows];   // results: written, read by who needs them
  uint64_t pre_full[kMaxRows], p2_done[kMaxRows];       // distillation
  __device__ void init(int team_warps) {
    for (int i = 0; i < kMaxSlots; i++) tc::mbar_init(&full[i], 1), tc::mbar_init(&empty[i], kConsWarps / kGroups);
    for (int i = 0; i < kMaxRows; i++) {
      tc::mbar_init(&part_full[i], kConsWarps);
      tc::mbar_init(&part_empty[i], team_warps);
      for (int j = 0; j < 2; j++) tc::mbar_init(&joined[i][j], 1);
      tc::mbar_init(&scal_full[i], 1);
      tc::mbar_init(&scal_empty[i], 1);
      tc::mbar_init(&pre_full[i], team_warps);
      tc::mbar_init(&p2_done[i], kConsWarps);
    }
    tc::fence_mbar_init();
  }
};

// A position in the ring: slot, and the parity of the slot's round.
struct RingPos {
  int slot = 0;
  uint32_t round = 0;
  __device__ __forceinline__ void skip(int n, int n_slots) {
    slot += n;
    while (slot >= n_slots) slot -= n_slots, round ^= 1;
  }
};

constexpr int kSmemMax = 227 * 1024;

// SMs and bytes of L2 of the current device
int sm_count();
int64_t l2_bytes();

// Clusters of cs CTAs of this kernel that the device holds at once.
int max_clusters(const void* kernel, int cs, int smem, int* out);

// CTAs per row for n rows of nv vectors: several only where every row has its cluster at once
// (a cluster that takes row after row waits for its slowest CTA at each), and where the time
// that the shorter parts save is more than joining them costs.
//   join_us(cs): what a cluster of cs CTAs costs besides, in microseconds.
template <typename F>
int pick_cluster(const void* kernel, int32_t n, int64_t nv, int smem, F join_us, int* cs) {
  *cs = 1;
  if (int st = set_smem_limit(kernel, kSmemMax)) return st;
  double best = (double)nv * 16e-3 / 65;   // a CTA streams a row at about 65 KB/us
  for (int c = 2; c <= kMaxCluster && (int64_t)n * c <= sm_count(); c *= 2) {
    const double t = (double)nv * 16e-3 / 65 / c + join_us(c);
    if (t >= best) continue;
    int held = 0;
    if (int st = max_clusters(kernel, c, smem, &held)) return st;
    if (n <= held) best = t, *cs = c;
  }
  return OCTO_OK;
}

// Launches kernel(p), which calls wait_for_predecessor, with `grid` CTAs in clusters of cs.
int launch_overlapped(const void* kernel, const void* p, int grid, int block, int cs, int smem, cudaStream_t s);

// Launches kernel(p) on n rows: a cluster of cs CTAs for each, but no more than the device holds.
int launch_ring_raw(const void* kernel, const void* p, int32_t n, int cs, int smem, cudaStream_t s);
template <typename P>
int launch_ring(const void* kernel, const P& p, int32_t n, int cs, int smem, cudaStream_t s) {
  return launch_ring_raw(kernel, &p, n, cs, smem, s);
}

}  // namespace rows
}  // namespace octo
