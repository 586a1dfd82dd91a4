// Chunk plans, and the entry points of the chunk attention.
//
// Octopus project page, "Architecture & Co-Design" item 01 (Runtime): a turn extends a cursor
// over the pages it shares; item 02: mounted spans are read in place.  A chunk plan is to
// several new tokens of a cursor what a decode plan is to one.  It lists, per cursor, the
// context in blocks of 64 keys, once for all of the cursor's tiles (without a window a tile's
// blocks are a prefix of them; under one, each tile lists the few that it sees).  What several
// cursors next to each other share, common ancestors up to the same point, is listed once for
// all of them: their rows, next to each other too, make tiles of their own for it, so that the
// prefix of a tree's branches is read once and not once a branch.  The tiles' block lists are
// cut into pieces for the CTAs.  The plan is built on the host: a step's plan serves every layer
// of a model, and its size is that of the contexts' page lists (256 cursors of 26,000 tokens: 1.7
// ms, where their decode plan takes 8).

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <new>
#include <queue>

#include "chunk.h"
#include "row_ring.cuh"

namespace octo {
namespace {

// Rows [row0, row0 + rows) of the plan, and blocks that some of them sees.  Of one cursor: tokens
// from own index t0 on (under a window at positions own index + shift, no mount among them).  Or of
// several cursors next to each other, with blocks of common ancestors, which all of them see (t0 = 0).
struct ChunkTile {
  int32_t row0, rows, t0, shift;
  int32_t blk0, n_blk;
};

// Keys per block: 64 where pages make up 64 keys or are made up of them, so that a block is 64
// rows of a tensor-core tile; else a page.
int32_t block_width(int32_t P) { return (P % 64 == 0 || (P >= 16 && 64 % P == 0)) ? 64 : P; }

// The first `fork` tokens of segment seg, and its mounts among the first n_mounts up to there.
struct Level {
  int32_t seg, fork, n_mounts;
  bool operator==(const Level& o) const { return seg == o.seg && fork == o.fork && n_mounts == o.n_mounts; }
};

struct Builder {
  const octo_pool_s* pool;
  int32_t P, W, n_sink;
  bool windowed;
  std::vector<ChunkBlock> out;

  // tokens [a, b) of segment s; own: they are the cursor's own; from: see ChunkBlock
  void span(int32_t s, int32_t a, int32_t b, bool own, int32_t from) {
    const Segment& g = pool->segs[s];
    for (int32_t c = a / W * W; c < b; c += W) {
      const int32_t end = std::min(b, c + W);
      for (int32_t t = std::max(a, c); t < end;) {
        int32_t e = end, seen = from;
        if (windowed) {
          // the run from t on: positions rise by one, sinks or not
          const bool sink = g.pos[t] < n_sink;
          if (g.pos[end - 1] - g.pos[t] != end - 1 - t || (sink && g.pos[end - 1] >= n_sink))
            for (e = t + 1; e < end && g.pos[e] == g.pos[e - 1] + 1 && (g.pos[e] < n_sink) == sink;) e++;
          seen = sink ? kSinkPos : g.pos[t] - (t - c);
        }
        ChunkBlock k;
        const int32_t p0 = c / P;
        for (int i = 0; i < 4; i++) k.page[i] = g.pages[std::min<size_t>(p0 + i, g.pages.size() - 1)];
        k.slot0 = c % P;
        k.own0 = own ? c : kFarOwn;
        k.seen = seen;
        k.lo = (uint16_t)(t - c);
        k.hi = (uint16_t)(e - c);
        out.push_back(k);
        t = e;
      }
    }
  }

  // what a child sees of its parent: the mounts it held by then, and its first tokens
  void ancestor(const Level& l) {
    const std::vector<int32_t>& mounts = pool->segs[l.seg].mounts;
    for (int32_t i = 0; i < l.n_mounts; i++) {
      const MountRec& m = pool->mounts[mounts[i]];
      if (m.m <= l.fork) span(m.producer, m.a, m.b, false, 0);
    }
    span(l.seg, 0, l.fork, false, 0);
  }
};

Level level_of(const octo_pool_s* pool, int32_t child) {
  const Segment& c = pool->segs[child];
  Level l{c.parent, c.fork, 0};
  for (int32_t id : pool->segs[c.parent].mounts) l.n_mounts += pool->mounts[id].created < c.created;   // in order of creation
  return l;
}

// A cursor with rows and what it sees besides its own segment, from the root on.
struct Path {
  int32_t cursor;
  std::vector<Level> levels;
  size_t first;                  // the levels before it are in shared tiles
  std::vector<int32_t> shared;   // those tiles
};

// Finds the runs of cursors with common levels.  share(from, to, l0, l1): makes tiles of the paths
// [from, to) with their common levels [l0, l1) and notes it in each path that got one.
template <typename F>
struct Sharing {
  const octo_pool_s* pool;
  std::vector<Path>& paths;
  F share;
  void range(size_t from, size_t to, size_t l0, size_t depth) {
    if (to - from < 2) return;
    size_t l1 = depth;
    auto same = [&](size_t i, size_t l) {
      return l < paths[i].levels.size() && l < paths[from].levels.size() && paths[i].levels[l] == paths[from].levels[l];
    };
    auto all_same = [&] {
      for (size_t i = from; i < to; i++)
        if (!same(i, l1)) return false;
      return true;
    };
    while (all_same()) l1++;
    if (l1 > l0) share(from, to, l0, l1);
    // runs whose next level, and what is left to share before it, are the same
    for (size_t i = from; i < to;) {
      size_t e = i + 1;
      auto alike = [&](size_t k) {
        return paths[k].first == paths[i].first && l1 < paths[i].levels.size() && l1 < paths[k].levels.size() &&
               paths[k].levels[l1] == paths[i].levels[l1];
      };
      while (e < to && alike(e)) e++;
      range(i, e, std::max(l0, paths[i].first), l1);
      i = e;
    }
  }
};
template <typename F>
Sharing(const octo_pool_s*, std::vector<Path>&, F) -> Sharing<F>;

// Shared blocks that are worth tiles of their own: with fewer, the items and the partial results
// that these cost take longer than reading the blocks again (from L2 mostly).  At 4, 8 and 16, us, five
// new tokens of each cursor: one tree of six cursors behind 256 shared tokens 10.3, 7.1 and 7.1, 384:
// 11.9, 8.6 and 8.6, 512: 12.9, 13.5 and 10.1, 768: 10.0, 10.0 and 11.0; eight such trees, 256: 12.6, 16.1
// and 16.1, 512: 15.1, 15.1 and 18.7, 768: 15.6, 15.6 and 22.8; 32 with 700 tokens of their own, 256: 94,
// 78 and 78, 768: 90, 89 and 107.
constexpr int32_t kShareBlocks = 8;

// Visible (row, key) pairs of a tile's block.
int64_t block_pairs(const ChunkBlock& k, const ChunkTile& t, int32_t window) {
  const int32_t last = t.t0 + t.rows - 1;
  auto lo = [&](int32_t i) {
    return window ? std::max<int32_t>(k.lo, i + t.shift - window + 1 - k.seen) : k.seen <= i ? (int32_t)k.lo : (int32_t)k.hi;
  };
  auto hi = [&](int32_t i) { return std::min<int32_t>(k.hi, i - k.own0 + 1); };
  if (hi(t.t0) == k.hi && lo(t.t0) == k.lo && lo(last) == k.lo) return (int64_t)t.rows * (k.hi - k.lo);
  int64_t n = 0;
  for (int32_t i = t.t0; i <= last; i++) n += std::max(0, hi(i) - lo(i));
  return n;
}

// The cuts of a plan's tiles into work, in the order of the tiles and of the kv heads: of each
// (tile, kv head) the pieces, in blocks, and who takes them.
struct Cut {
  int32_t n, cta;
};
using Cuts = std::vector<std::vector<Cut>>;

// For the CUDA-core kernels, which give a piece a CTA: pieces of about `len` blocks, the length
// with the shortest makespan among those that fill the SMs 1, 2, ... times; a piece costs
// kPieceCost blocks more (its start, its queries, its results), a join kJoinCost once.
constexpr int kPieceCost = 5, kJoinCost = 4;
Cuts cut_evenly(const std::vector<ChunkTile>& tiles, int heads, int sms) {
  int32_t most = 1;
  for (const ChunkTile& t : tiles) most = std::max(most, t.n_blk);
  auto pieces = [&](int32_t len) {
    int64_t n = 0;
    for (const ChunkTile& t : tiles) n += (t.n_blk + len - 1) / len;
    return n * heads;
  };
  int32_t best = most;
  int64_t best_t = INT64_MAX;
  auto consider = [&](int32_t len) {
    // longest first, each to the SM that is free first
    std::vector<int32_t> lens;
    for (const ChunkTile& t : tiles)
      for (int32_t k = (t.n_blk + len - 1) / len, i = 0; i < k; i++) lens.push_back((t.n_blk - i + k - 1) / k + kPieceCost);
    std::sort(lens.begin(), lens.end(), std::greater<int32_t>());
    std::priority_queue<int64_t, std::vector<int64_t>, std::greater<int64_t>> q;
    for (int i = 0; i < sms; i++) q.push(0);
    int64_t end = 0;
    for (int32_t l : lens)
      for (int h = 0; h < heads; h++) {
        const int64_t t = q.top() + l;
        q.pop(), q.push(t);
        end = std::max(end, t);
      }
    end += lens.size() > tiles.size() ? kJoinCost : 0;
    if (end < best_t) best_t = end, best = len;
  };
  if (pieces(most) <= 24LL * sms) {   // else many waves: nothing to gain
    consider(most);
    for (int w = 1; w <= 6; w++) {
      // the shortest pieces of which w waves are enough
      int32_t lo = 1, hi = most;
      while (lo < hi) {
        const int32_t mid = lo + (hi - lo) / 2;
        if (pieces(mid) <= (int64_t)w * sms) hi = mid;
        else lo = mid + 1;
      }
      if (pieces(lo) <= (int64_t)w * sms) consider(lo);
    }
  }
  Cuts cuts;
  for (const ChunkTile& t : tiles) {
    const int32_t k = std::max(1, (t.n_blk + best - 1) / best);
    std::vector<Cut> c;
    for (int32_t i = 0; i < k; i++) c.push_back({(t.n_blk + i) / k, 0});
    cuts.insert(cuts.end(), heads, c);
  }
  return cuts;
}

// CTAs of a tensor-core kernel, each of which takes several pieces: one an SM, but no more than
// have kLeast blocks each.  A piece costs `change` blocks more.  (One cursor with 24 blocks a kv
// head: 8.9 us at pieces of 1 and 10.2 at pieces of 3.)
constexpr int kLeast = 1;
int cta_count(const std::vector<ChunkTile>& tiles, int heads, int sms, double change, double* total) {
  *total = 0;
  for (const ChunkTile& t : tiles) *total += heads * (t.n_blk + change);
  return (int)std::max(1.0, std::min((double)sms, *total / (kLeast + change)));
}

// One slot: all work in a row, cut into runs of equal cost, so that all CTAs end together.
constexpr double kStreamChange = 1.0;
constexpr int kWhole = 8;   // tiles that are all this short and few are not cut: joining them takes as long
Cuts cut_into_runs(const std::vector<ChunkTile>& tiles, int heads, int sms) {
  int32_t longest = 0;
  for (const ChunkTile& t : tiles) longest = std::max(longest, t.n_blk);
  if (longest <= kWhole && (int64_t)tiles.size() * heads <= sms) {
    Cuts whole;
    int32_t cta = 0;
    for (const ChunkTile& t : tiles)
      for (int h = 0; h < heads; h++) whole.push_back({{t.n_blk, cta++}});
    return whole;
  }
  double total = 0;
  const int ctas = cta_count(tiles, heads, sms, kStreamChange, &total);
  const double budget = (total + (ctas - 1) * kStreamChange) / ctas;   // a run's end cuts a tile: a piece more
  Cuts cuts;
  double at = 0;   // cost so far
  int32_t cta = 0, pieces = 0;
  for (const ChunkTile& t : tiles)
    for (int h = 0; h < heads; h++) {
      cuts.emplace_back();
      for (int32_t left = t.n_blk; left > 0;) {
        // what the CTA at hand has room for; a remainder of a block or two stays with it
        const double room = (cta + 1) * budget - at - kStreamChange;
        const bool last = cta + 1 == ctas;
        if (!last && room < 0.5 && pieces > 0) {
          cta++, pieces = 0;
          continue;
        }
        const int32_t take = last || room >= left - 2 ? left : std::max(1, (int32_t)(room + 0.5));
        cuts.back().push_back({take, cta});
        left -= take;
        pieces++;
        at += take + kStreamChange;
      }
    }
  return cuts;
}

constexpr int kPairBlocks = 6;

// Two slots: a tile's partial result is up to 128 KB, so tiles go whole, longest first, to the
// CTA with the least work, as long as that does not pass the average; what is left is cut to
// fill the CTAs up.  (512 tiles of 35 blocks on 152 CTAs: three whole ones each, 56 cut.)
constexpr double kPairChange = 7.0, kPartChange = 9.0;   // pieces cost 6 us more than their blocks of 0.83 us
Cuts cut_what_is_left(const std::vector<ChunkTile>& tiles, int heads, int sms) {
  double total = 0;
  const int ctas = cta_count(tiles, heads, sms, kPairChange, &total);
  Cuts cuts(tiles.size() * heads);
  std::vector<int32_t> order(cuts.size()), left;
  for (size_t i = 0; i < order.size(); i++) order[i] = (int32_t)i;
  auto blocks = [&](int32_t i) { return tiles[i / heads].n_blk; };
  std::stable_sort(order.begin(), order.end(), [&](int32_t x, int32_t y) { return blocks(x) > blocks(y); });
  std::vector<double> load(ctas, 0);
  using Item = std::pair<double, int32_t>;
  std::priority_queue<Item, std::vector<Item>, std::greater<Item>> q;
  for (int32_t c = 0; c < ctas; c++) q.push({0.0, c});
  for (int32_t i : order) {
    const Item c = q.top();
    const double t = c.first + blocks(i) + kPairChange;
    if (t > total / ctas + 1) {
      left.push_back(i);
      continue;
    }
    q.pop(), q.push({t, c.second});
    load[c.second] = t;
    cuts[i].push_back({blocks(i), c.second});
  }
  if (left.empty()) return cuts;
  // the level up to which the CTAs are filled: each takes a piece, and one more where a tile ends in it
  double rest = 0;
  for (int32_t i : left) rest += blocks(i) + kPartChange;
  double lo = 0, hi = total + kPartChange;
  for (int k = 0; k < 40; k++) {
    const double mid = (lo + hi) / 2;
    double room = 0;
    for (double l : load) room += std::max(0.0, mid - l - kPartChange);
    (room >= rest ? hi : lo) = mid;
  }
  int32_t c = 0;
  for (int32_t i : left)
    for (int32_t n = blocks(i); n > 0;) {
      while (c + 1 < ctas && hi - load[c] - kPartChange < 1.0) c++;
      const double room = hi - load[c] - kPartChange;
      const int32_t take = c + 1 == ctas || room >= n - 2 ? n : std::max(1, (int32_t)(room + 0.5));
      cuts[i].push_back({take, c});
      n -= take;
      load[c] += take + kPartChange;
    }
  return cuts;
}

template <typename T>
size_t place(size_t* at, const std::vector<T>& v) {
  const size_t o = *at;
  *at = align_up(o + v.size() * sizeof(T), 256);
  return o;
}

// the pool's device status word, made on first use
int ensure_status(octo_pool_s* pool) {
  if (!pool->d_status) {
    OCTO_CUDA(cudaMalloc(&pool->d_status, sizeof(int32_t) * 4));
    OCTO_CUDA(cudaMemset(pool->d_status, 0, sizeof(int32_t) * 4));
  }
  return OCTO_OK;
}

int build(octo_pool_s* pool, const octo_cursor_t* cursors, const int32_t* n_new, int32_t n, int32_t Hq,
          int32_t window, int32_t n_sink, cudaStream_t s, octo_plan_t* out) {
  const octo_pool_desc& d = pool->desc;
  std::unique_ptr<octo_plan_s> pl(new octo_plan_s());
  std::unique_ptr<ChunkPlan> cp(new ChunkPlan());
  cp->Hq = Hq;
  cp->G = Hq / d.n_kv_heads;
  cp->width = block_width(d.page_size);
  cp->tokens = std::max(1, 128 / cp->G);
  cp->tc = chunk_tc_supported(d, cp->width);
  cp->row0.resize((size_t)n + 1, 0);
  int64_t rows = 0;
  int32_t top = 0;   // the largest position of a row
  for (int32_t i = 0; i < n; i++) {
    rows += n_new[i];
    if (rows > INT32_MAX / 2) return OCTO_EINVAL;
    cp->row0[i + 1] = (int32_t)rows;
    if (n_new[i]) top = std::max(top, pool->segs[cursors[i]].pos.back());
  }
  if (top >= kMaxPos) return OCTO_ENOTSUP;
  cp->window = window > top ? 0 : window;   // sees everything

  // Tiles have the rows of one 128-row tile, or of two where a chunk is longer and, for the tensor
  // cores, the work is more than kPairBlocks blocks an SM.  (Less of it is sooner done in twice as
  // many pieces: four chunks of 80 tokens under a window of 1,000 take 15 us so and 20 in pairs;
  // 22 either way at 160 tokens; four of 40 behind 4,096 tokens 22 and 18.)
  const int sms = std::max(1, rows::sm_count()), heads = d.n_kv_heads;
  int32_t most_new = 0;
  int64_t pair_blocks = 0;
  for (int32_t c = 0; c < n; c++) {
    if (!n_new[c]) continue;
    most_new = std::max(most_new, n_new[c]);
    const int32_t seen = pool->segs[cursors[c]].pos.back() + 1;   // keys, about
    pair_blocks += (int64_t)((n_new[c] + 2 * cp->tokens - 1) / (2 * cp->tokens)) *
                   ((cp->window ? std::min(seen, cp->window + 2 * cp->tokens) : seen) / cp->width + 1) * heads;
  }
  const int32_t cap = most_new > cp->tokens && (!cp->tc || pair_blocks > (int64_t)kPairBlocks * sms) ? 2 * cp->tokens : cp->tokens;
  Builder b{pool, d.page_size, cp->width, cp->window ? n_sink : 0, cp->window > 0, {}};
  std::vector<ChunkBlock> blocks;
  std::vector<ChunkTile> tiles;
  std::vector<int32_t> row_pos((size_t)rows);
  int64_t pairs = 0;
  auto add_pairs = [&](const ChunkTile& t) {
    for (int32_t i = 0; i < t.n_blk; i++) pairs += block_pairs(blocks[t.blk0 + i], t, cp->window);
  };

  // tiles of several cursors
  std::vector<Path> paths;
  for (int32_t c = 0; c < n; c++) {
    if (!n_new[c]) continue;
    paths.push_back({c, {}, 0, {}});
    for (int32_t x = cursors[c]; pool->segs[x].parent >= 0; x = pool->segs[x].parent)
      paths.back().levels.push_back(level_of(pool, x));
    std::reverse(paths.back().levels.begin(), paths.back().levels.end());
  }
  if (!cp->window) {
    Sharing sh{pool, paths, [&](size_t from, size_t to, size_t l0, size_t l1) {
      // cursors [from, to) of `paths` and their common levels [l0, l1)
      b.out.clear();
      for (size_t l = l0; l < l1; l++) b.ancestor(paths[from].levels[l]);
      if ((int32_t)b.out.size() < kShareBlocks) return false;
      const int32_t blk0 = (int32_t)blocks.size();
      bool any = false;
      for (size_t i = from; i < to;) {
        size_t e = i;
        int32_t tokens = 0;
        while (e < to && tokens + n_new[paths[e].cursor] <= cap) tokens += n_new[paths[e++].cursor];
        if (e - i < 2) {
          i = std::max(e, i + 1);
          continue;
        }
        if (!any) blocks.insert(blocks.end(), b.out.begin(), b.out.end());
        any = true;
        ChunkTile t = {};
        t.row0 = cp->row0[paths[i].cursor];
        t.rows = tokens;
        t.blk0 = blk0;
        t.n_blk = (int32_t)b.out.size();
        add_pairs(t);
        for (; i < e; i++) {
          paths[i].shared.push_back((int32_t)tiles.size());
          paths[i].first = l1;
        }
        tiles.push_back(t);
      }
      return any;
    }};
    sh.range(0, paths.size(), 0, 0);
  }
  const size_t n_shared = tiles.size();
  std::vector<const Path*> path_of;   // of the tiles from n_shared on

  std::vector<int32_t> from, cut;
  for (const Path& path : paths) {
    const int32_t c = path.cursor;
    const Segment& g = pool->segs[cursors[c]];
    const int32_t first = g.len - n_new[c];
    std::copy(g.pos.begin() + first, g.pos.end(), row_pos.begin() + cp->row0[c]);
    // the rest of the cursor's context, in the order in which its rows come to see it, and from
    // which of its segment's tokens on they do
    b.out.clear();
    for (size_t l = path.first; l < path.levels.size(); l++) b.ancestor(path.levels[l]);
    from.assign(b.out.size(), 0);
    cut.clear();
    int32_t next = 0;
    auto own_from = [&] {
      while (from.size() < b.out.size()) from.push_back(b.out[from.size()].own0 + b.out[from.size()].lo);
    };
    for (int32_t id : g.mounts) {
      const MountRec& m = pool->mounts[id];
      if (m.m > g.len - 1) continue;
      // the own tokens before the mount go first: what comes to be seen later is listed later.  Under
      // a window their block is cut there, where positions jump; without one it goes as a whole, the
      // tokens behind the mount being hidden from the rows before them
      const int32_t upto = cp->window ? m.m : std::min(g.len, (m.m + b.W - 1) / b.W * b.W);
      if (upto > next) {
        b.span(cursors[c], next, upto, true, 0);
        next = upto;
      }
      own_from();
      b.span(m.producer, m.a, m.b, false, m.m);
      from.resize(b.out.size(), m.m);
      if (m.m > first && cp->window) cut.push_back(m.m);
    }
    if (next < g.len) b.span(cursors[c], next, g.len, true, 0);
    own_from();
    cut.push_back(g.len);
    const int32_t base = (int32_t)blocks.size();
    if (!cp->window) blocks.insert(blocks.end(), b.out.begin(), b.out.end());
    // tiles; under a window without a mount inside, so that their positions rise by one
    size_t seen = 0;
    for (int32_t t = first, k = 0; t < g.len;) {
      while (cut[k] <= t) k++;
      ChunkTile tile = {};
      tile.row0 = cp->row0[c] + t - first;
      tile.t0 = t;
      tile.rows = std::min(cap, cut[k] - t);
      tile.shift = g.pos[t] - t;
      const int32_t last = t + tile.rows - 1;
      while (seen < b.out.size() && from[seen] <= last) seen++;
      if (cp->window) {
        tile.blk0 = (int32_t)blocks.size();
        for (size_t i = 0; i < seen; i++) {
          const ChunkBlock& x = b.out[i];
          if (x.seen + x.hi - 1 > g.pos[t] - cp->window) blocks.push_back(x);
        }
        tile.n_blk = (int32_t)blocks.size() - tile.blk0;
      } else {
        tile.blk0 = base;
        tile.n_blk = (int32_t)seen;
      }
      add_pairs(tile);
      tiles.push_back(tile);
      path_of.push_back(&path);
      t += tile.rows;
    }
    if (blocks.size() > (size_t)INT32_MAX / 2) return OCTO_EINVAL;
  }

  // the work, in pieces of the tiles' blocks, and the joins of what has several
  for (const ChunkTile& t : tiles) cp->max_rows = std::max(cp->max_rows, t.rows);
  std::vector<int32_t> cta_work, refs;
  const Cuts cuts = !cp->tc ? cut_evenly(tiles, heads, sms)
                    : cp->max_rows > cp->tokens ? cut_what_is_left(tiles, heads, sms) : cut_into_runs(tiles, heads, sms);
  std::vector<ChunkWork> work;
  std::vector<int32_t> cta_of;   // of each piece
  std::vector<ChunkJoin> joins;
  std::vector<std::pair<size_t, size_t>> work_of(cuts.size());   // [first, end) of each (tile, kv head)'s
  int32_t longest = 0;
  for (size_t i = 0; i < tiles.size(); i++) {
    const ChunkTile& t = tiles[i];
    longest = std::max(longest, t.n_blk);
    for (int32_t g = 0; g < heads; g++) {
      const std::vector<Cut>& cut = cuts[i * heads + g];
      const bool partial = cut.size() > 1 || i < n_shared || !path_of[i - n_shared]->shared.empty();
      work_of[i * heads + g] = {work.size(), work.size() + cut.size()};
      for (int32_t at = t.blk0, k = 0; k < (int32_t)cut.size(); at += cut[k++].n) {
        work.push_back({t.row0, t.rows, t.t0, t.shift, at, cut[k].n, g, partial ? (int32_t)cp->n_part : -1});
        cta_of.push_back(cut[k].cta);
        if (partial) cp->n_part += (int64_t)t.rows * cp->G;
        if (cp->n_part > INT32_MAX) return OCTO_EINVAL;
      }
      if (i < n_shared || !partial) continue;
      const int32_t ref0 = (int32_t)refs.size();
      auto add = [&](size_t tile) {
        const auto& w = work_of[tile * heads + g];
        for (size_t x = w.first; x < w.second; x++) refs.push_back(work[x].part + (t.row0 - tiles[tile].row0) * cp->G);
      };
      for (int32_t x : path_of[i - n_shared]->shared) add(x);
      add(i);
      const int32_t n_refs = (int32_t)refs.size() - ref0;
      joins.push_back({t.row0, t.rows, g, ref0, n_refs});
      cp->max_join_rows = std::max(cp->max_join_rows, t.rows);
      cp->max_refs = std::max(cp->max_refs, n_refs);
    }
  }
  if (cp->tc) {
    // by CTA
    cta_work.assign(1, 0);
    for (int32_t c : cta_of) {
      if ((size_t)c + 2 > cta_work.size()) cta_work.resize(c + 2, 0);
      cta_work[c + 1]++;
    }
    for (size_t c = 1; c < cta_work.size(); c++) cta_work[c] += cta_work[c - 1];
    std::vector<ChunkWork> sorted(work.size());
    std::vector<int32_t> next(cta_work);
    for (size_t i = 0; i < work.size(); i++) sorted[next[cta_of[i]]++] = work[i];
    work.swap(sorted);
  } else {
    std::stable_sort(work.begin(), work.end(), [](const ChunkWork& x, const ChunkWork& y) { return x.n > y.n; });
    for (const ChunkWork& w : work)
      for (int x = 1; x <= 8; x++) cp->simt_ctas[x] += ((int64_t)w.rows * cp->G + 16 * x - 1) / (16 * x);
  }
  if (work.size() > (size_t)INT32_MAX || joins.size() > (size_t)INT32_MAX) return OCTO_EINVAL;
  cp->n_work = (int32_t)work.size();
  cp->n_joins = (int32_t)joins.size();
  cp->n_ctas = cp->tc ? (int32_t)cta_work.size() - 1 : 0;

  // what octo_plan_copy_out gives of a chunk plan: its cursors, rows, positions and tiles
  std::vector<int32_t> order(cursors, cursors + n), t_seg, t_t0, t_rows, none(std::max((size_t)d.num_pages, tiles.size()) + 1, 0);
  for (size_t i = n_shared; i < tiles.size(); i++) {
    t_seg.push_back(cursors[path_of[i - n_shared]->cursor]);
    t_t0.push_back(tiles[i].t0), t_rows.push_back(tiles[i].rows);
  }

  // what the verification of drafted tokens goes by
  std::vector<int32_t> drafted;
  cp->live.assign((size_t)n + 1, 0);
  for (int32_t c = 0; c < n; c++) {
    cp->live[c + 1] = cp->live[c] + (n_new[c] > 0);
    for (int32_t r = cp->row0[c]; r + 1 < cp->row0[c + 1]; r++) drafted.push_back(r);
  }

  // device arrays: one allocation, one copy
  size_t at = 0;
  const size_t o_blk = place(&at, blocks), o_work = place(&at, work), o_cta = place(&at, cta_work), o_join = place(&at, joins), o_ref = place(&at, refs),
               o_pos = place(&at, row_pos), o_row0 = place(&at, cp->row0),
               o_order = place(&at, order), o_seg = place(&at, t_seg), o_t0 = place(&at, t_t0), o_rows = place(&at, t_rows),
               o_none = place(&at, none), o_drafted = place(&at, drafted), o_live = place(&at, cp->live);
  std::vector<char> stage(std::max<size_t>(at, 256));
  auto put = [&](size_t o, const auto& v) {
    if (!v.empty()) std::memcpy(stage.data() + o, v.data(), v.size() * sizeof(v[0]));
  };
  put(o_blk, blocks), put(o_work, work), put(o_cta, cta_work), put(o_join, joins), put(o_ref, refs), put(o_pos, row_pos), put(o_row0, cp->row0);
  put(o_order, order), put(o_seg, t_seg), put(o_t0, t_t0), put(o_rows, t_rows), put(o_none, none), put(o_drafted, drafted), put(o_live, cp->live);
  if (int st = ensure_status(pool)) return st;
  OCTO_CUDA(cudaGetDevice(&pl->device));
  pl->pool = pool;
  pl->last_stream = s;
  pl->num_pages = d.num_pages;
  void* buf = nullptr;
  OCTO_CUDA(cudaMallocAsync(&buf, stage.size(), s));
  pl->allocs.push_back(buf);
  char* base = static_cast<char*>(buf);
  cp->blocks = reinterpret_cast<ChunkBlock*>(base + o_blk);
  cp->work = reinterpret_cast<ChunkWork*>(base + o_work);
  cp->cta_work = reinterpret_cast<int32_t*>(base + o_cta);
  cp->joins = reinterpret_cast<ChunkJoin*>(base + o_join);
  cp->refs = reinterpret_cast<int32_t*>(base + o_ref);
  cp->drafted = reinterpret_cast<int32_t*>(base + o_drafted);
  cp->d_live = reinterpret_cast<int32_t*>(base + o_live);
  pl->row_pos = reinterpret_cast<int32_t*>(base + o_pos);
  pl->seg_row_base = reinterpret_cast<int32_t*>(base + o_row0);
  pl->seg_order = reinterpret_cast<int32_t*>(base + o_order);
  pl->tile_seg = reinterpret_cast<int32_t*>(base + o_seg);
  pl->tile_t0 = reinterpret_cast<int32_t*>(base + o_t0);
  pl->tile_rows = reinterpret_cast<int32_t*>(base + o_rows);
  pl->tile_off = pl->page_off = reinterpret_cast<int32_t*>(base + o_none);   // no entries
  std::memset(&pl->info, 0, sizeof(pl->info));
  pl->info.n_rows = rows;
  pl->info.n_tiles = (int64_t)path_of.size();
  pl->info.n_segments = n;
  pl->info.pairs = pairs;
  pl->info.bm = cap;
  pl->info.page_size = d.page_size;
  pl->info.max_tile_entries = longest;
  pl->info.is_decode = 2;
  pl->max_succ = 1;
  pl->chunk = std::move(cp);
  int st = cuda_status(cudaMemcpyAsync(buf, stage.data(), stage.size(), cudaMemcpyHostToDevice, s));
  if (st == OCTO_OK) st = cuda_status(cudaStreamSynchronize(s));   // the staging buffer goes, other streams may use the plan
  if (st != OCTO_OK) {
    octo_plan_destroy(pl.release());
    return st;
  }
  *out = pl.release();
  return OCTO_OK;
}

size_t part_floats(const octo_plan_s* p) {
  return (size_t)p->chunk->n_part * p->pool->desc.head_dim;
}

}  // namespace
}  // namespace octo

extern "C" {

int octo_chunk_plan(octo_pool_t pool, const octo_cursor_t* cursors, const int32_t* n_new, int32_t n, int32_t Hq,
                    int32_t window, int32_t n_sink, void* stream, octo_plan_t* out) {
  octo::NvtxRange nv("octo_chunk_plan");
  if (!pool || !out || n < 0 || (n > 0 && (!cursors || !n_new))) return OCTO_EINVAL;
  if (Hq <= 0 || Hq % pool->desc.n_kv_heads || Hq > 65535) return OCTO_EINVAL;
  if (window < 0 || n_sink < 0 || (!window && n_sink)) return OCTO_EINVAL;
  if (Hq / pool->desc.n_kv_heads > 128) return OCTO_ENOTSUP;
  for (int32_t i = 0; i < n; i++) {
    const int32_t c = cursors[i];
    if (c < 0 || c >= (int32_t)pool->segs.size() || pool->segs[c].freed) return OCTO_EINVAL;
    if (n_new[i] < 0 || n_new[i] > pool->segs[c].len) return OCTO_EINVAL;
  }
  try {
    return octo::build(pool, cursors, n_new, n, Hq, window, n_sink, (cudaStream_t)stream, out);
  } catch (const std::bad_alloc&) {
    return OCTO_ENOMEM;
  }
}

size_t octo_chunk_attn_workspace_size(octo_plan_t plan) {
  if (!plan || !plan->chunk) return 0;
  const size_t rows = (size_t)plan->chunk->n_part;
  return rows ? octo::align_up(octo::part_floats(plan) * sizeof(float), 256) + rows * 2 * sizeof(float) : 0;
}

int octo_chunk_attn(octo_plan_t plan, const void* q, const void* k_pool, const void* v_pool, void* out, float* lse,
                    float scale, void* ws, size_t ws_bytes, void* stream) {
  octo::NvtxRange nv("octo_chunk_attn");
  if (!plan || !plan->chunk) return OCTO_EINVAL;
  // the running maximum is that of the unscaled scores, and hidden ones are -inf times the scale
  if (!(scale >= 1e-30f) || !std::isfinite(scale)) return OCTO_EINVAL;
  int dev = 0;
  OCTO_CUDA(cudaGetDevice(&dev));
  if (dev != plan->device) return OCTO_EINVAL;
  if (plan->info.n_rows == 0) return OCTO_OK;
  octo::ChunkArgs a;
  a.q = q;
  a.k = k_pool ? k_pool : plan->pool->desc.k_pool;
  a.v = v_pool ? v_pool : plan->pool->desc.v_pool;
  a.out = out;
  a.lse = lse;
  a.scale = scale;
  if (!q || !out || !a.k || !a.v) return OCTO_EINVAL;
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)a.k | (uintptr_t)a.v | (uintptr_t)lse) & 15) return OCTO_EINVAL;
  const size_t need = octo_chunk_attn_workspace_size(plan);
  if (need && (!ws || ws_bytes < need || ((uintptr_t)ws & 15))) return OCTO_EINVAL;
  a.part = static_cast<float*>(ws);
  a.part_ml = need ? reinterpret_cast<float*>(static_cast<char*>(ws) + octo::align_up(octo::part_floats(plan) * sizeof(float), 256)) : nullptr;
  cudaStream_t s = (cudaStream_t)stream;
  plan->last_stream = s;
  if (int st = plan->chunk->tc ? octo::chunk_tc(plan, a, s) : octo::chunk_simt(plan, a, s)) return st;
  return plan->chunk->n_joins ? octo::chunk_join(plan, a, s) : OCTO_OK;
}

}  // extern "C"
