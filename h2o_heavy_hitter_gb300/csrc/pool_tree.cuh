// Attention of drafted tokens: the list of tiles that CTAs share, and what a row of a
// tree may attend to. (The kernels are in pool_prefix.cu and pool_tree.cu.)
//
// Where a head has at most 128 rows, each half of a CTA's softmax warps is a worker with a share of
// its own, and the CTA's tiles are those of both in turn; else the CTA is one worker.
//
// Entry b of a call has nodes[b] drafts, the last tokens of its sequence; node t attends to
// the prefix, to the tokens before the drafts, to the nodes of its branch and itself. Units are
// (entry, key head, block of two row tiles); row (t, g) of a head is node t of query head g of
// the head's group. A unit's tiles of 128 keys are the prefix's, then the sequence's own.
#pragma once

#include "pool_tiles.cuh"
#include "rotary.h"

#ifdef __CUDACC__
namespace h2o {

struct TreeEntry {
  int seq, len, nodes;  // nodes 0: nothing to do
  int tiles;            // of a unit
  int blocks;           // units of a head
};

// What the block finds out about the list before it begins, in shared memory.
struct TreeList {
  uint32_t skip[kPoolMaxList / 32];  // refused entries
  // of each worker: its share of all tiles, the entry in which that begins, and units x tiles before the
  // entry. The first has the larger share.
  int64_t at[2], end[2];
  int worker[2], b[2], cum[2];
  TreeEntry e[2];
};

// bad: what there is to report.
__device__ __forceinline__ TreeEntry tree_entry(const AttendParams& p, int b, int ptiles, int* bad) {
  const PoolView& v = p.a.v;
  TreeEntry e{};
  *bad = 0;
  e.seq = p.a.seqs[b];
  if (e.seq < 0 || e.seq >= v.seqs || e.seq == p.a.prefix) {
    if (e.seq != -1) *bad = kErrBadList;
    e.seq = -1;
    return e;
  }
  const int refused = __ldcg(v.refused + e.seq);  // (its last tokens are no drafts)
  int nodes = p.t.lens ? p.t.lens[b] : p.t.T;
  e.len = checked_length(v, e.seq, false);
  if (e.len < 0) *bad = kErrBadState;
  if (e.len < 0 || refused) return e;
  if (nodes < 0 || nodes > p.t.T) {
    *bad = kErrBadLength;
    nodes = nodes < 0 ? 0 : p.t.T;
  }
  if (nodes > e.len) {  // more drafts than tokens
    *bad = kErrBadLength;
    return e;
  }
  e.nodes = nodes;
  if (nodes == 0) return e;
  e.tiles = ptiles + key_tiles(e.len);
  e.blocks = (nodes + 2 * p.s.per_tile - 1) / (2 * p.s.per_tile);
  return e;
}

// Unit u and tile kt of tile `at` of an entry's: {u / blocks, u % blocks, kt}.
static __device__ __noinline__ int3 tree_place(int64_t at, int tiles, int blocks) {
  // (a division of 64 bits takes five times as long)
  const int u = at >> 32 ? static_cast<int>(at / tiles) : static_cast<int>(static_cast<uint32_t>(at) / static_cast<uint32_t>(tiles));
  const int h = u / blocks;
  return make_int3(h, u - h * blocks, static_cast<int>(at - static_cast<int64_t>(u) * tiles));
}

// Fills the list's summary for workers cta and (of two) cta + gridDim.x. Blockwide; `bits`: 4 KB. Block 0
// sets the error word; every one leaves what the joining kernel reads of its workers. Every call begins with this: an
// entry is read once, and its threads meet three times.
constexpr int kTreeThreads = 384;  // at least
constexpr int kTreePer = (kPoolMaxList + kTreeThreads - 1) / kTreeThreads;

__device__ __forceinline__ void tree_list(const AttendParams& p, int workers, int ptiles, int cta, TreeList& list,
                                          uint32_t* bits, int* wsum) {
  const bool report = cta == 0;
  const PoolView& v = p.a.v;
  const int tid = threadIdx.x, nt = blockDim.x, n = p.t.n, lane = tid & 31, warp = tid >> 5;
  const int per = (n + nt - 1) / nt, b0 = tid * per;
  TreeEntry e[kTreePer];
  int bad[kTreePer] = {};
#pragma unroll
  for (int i = 0; i < kTreePer; ++i)
    if (i < per && b0 + i < n) e[i] = tree_entry(p, b0 + i, ptiles, &bad[i]);
  // entries named before: looked for one by one only where a hashed bit says that there may be some
  bool seen = false;
  if (n > 1) {
#pragma unroll 1
    for (int i = tid; i < 1024; i += nt) bits[i] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTreePer; ++i)
      if (i < per && b0 + i < n && e[i].seq >= 0)
        seen |= (atomicOr(&bits[(e[i].seq >> 5) & 1023], 1u << (e[i].seq & 31)) >> (e[i].seq & 31)) & 1u;
  }
  if (tid < kPoolMaxList / 32) list.skip[tid] = 0;
  if (__syncthreads_or(seen)) {
#pragma unroll 1
    for (int b = b0; b < min(n, b0 + per); ++b) {
      const int s = p.a.seqs[b];
      if (s < 0) continue;
#pragma unroll 1
      for (int j = 0; j < b; ++j)
        if (p.a.seqs[j] == s) {
          if (report) atomicOr(v.err, kErrBadList);
          atomicOr(&list.skip[b >> 5], 1u << (b & 31));
          break;
        }
    }
    __syncthreads();
  }
  int weight[kTreePer], mine = 0;  // tiles of an entry's units of one head
#pragma unroll
  for (int i = 0; i < kTreePer; ++i) {
    const int b = b0 + i;
    const bool in = i < per && b < n && !((list.skip[b >> 5] >> (b & 31)) & 1u);
    weight[i] = in ? e[i].tiles * e[i].blocks : 0;
    mine += weight[i];
    if (report && in && bad[i]) atomicOr(v.err, bad[i]);  // (not of one that was named before)
  }
  int at = mine;  // inclusive over the warp, then over the block
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, at, off);
    if (lane >= off) at += y;
  }
  if (lane == 31) wsum[warp] = at;
  __syncthreads();
  const int sum = lane < nt / 32 ? wsum[lane] : 0;
  const int total = __reduce_add_sync(0xffffffffu, sum);
  at += __reduce_add_sync(0xffffffffu, lane < warp ? sum : 0) - mine;
  const int64_t all = static_cast<int64_t>(total) * p.s.heads;
  // lanes 0 .. 3 of every warp: where each worker's share begins and ends
  int64_t edge = 0;
  if (lane < 2 * workers) edge = share_begin(all, p.s.grid, cta + (lane >> 1) * gridDim.x + (lane & 1));
  int64_t begin[2], end[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    begin[i] = __shfl_sync(0xffffffffu, edge, 2 * i);
    end[i] = __shfl_sync(0xffffffffu, edge, 2 * i + 1);
  }
  const bool swap = workers == 2 && end[1] - begin[1] > end[0] - begin[0];
  if (tid < workers) {
    if ((tid ? end[1] - begin[1] : end[0] - begin[0]) == 0)
      p.w.cut[cta + tid * gridDim.x] = TreeCut{};
    const int slot = tid ^ swap;
    list.worker[slot] = cta + tid * gridDim.x;
    list.at[slot] = tid ? begin[1] : begin[0];
    list.end[slot] = tid ? end[1] : end[0];
  }
#pragma unroll
  for (int i = 0; i < kTreePer; ++i) {
    const int b = b0 + i;
    if (i >= per || b >= n) break;
    const int64_t lo = static_cast<int64_t>(at) * p.s.heads, hi = lo + static_cast<int64_t>(weight[i]) * p.s.heads;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k < workers && begin[k] >= lo && begin[k] < hi) {
        list.b[k ^ swap] = b;
        list.cum[k ^ swap] = at;
        list.e[k ^ swap] = e[i];
      }
    // the entry in which a worker's share ends: whether it leaves a unit there that it began
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k < workers && begin[k] < end[k] && end[k] > lo && end[k] <= hi) {
        const int worker = cta + k * gridDim.x;
        const int3 x = tree_place(end[k] - 1 - lo, e[i].tiles, e[i].blocks);  // head, block, tile
        const int64_t first = end[k] - 1 - x.z, behind = first + e[i].tiles;
        TreeCut cut{};
        if (first >= begin[k] && behind > end[k]) {
          cut.pieces = owner(behind - 1, all, p.s.grid) - worker + 1;
          cut.b = b;
          cut.h = x.x;
          cut.node = x.y * 2 * p.s.per_tile;
          cut.nodes = e[i].nodes;
        }
        p.w.cut[worker] = cut;
      }
    at += weight[i];
  }
}

// Entry b, or the next one that has tiles, which is then b. (What few steps of a walk take is out of line:
// six roles walk at once, and with all in line the kernels' 170 KB of code missed the instruction cache.)
static __device__ __noinline__ TreeEntry tree_next_entry(const AttendParams& p, const TreeList& list, int ptiles, int b,
                                                         int* found) {
  TreeEntry e;
  for (;; ++b) {
    int reported;
    e = tree_entry(p, b, ptiles, &reported);
    if (e.tiles && !((list.skip[b >> 5] >> (b & 31)) & 1u)) break;
  }
  *found = b;
  return e;
}

// A walk along one worker's share of the units.
struct TreeWalk {
  const AttendParams& p;
  const TreeList& list;
  int plen, ptiles, slot;
  int64_t at, end;
  // the unit
  bool two;
  int b, h, blk, kt0, kt1;
  TreeEntry e;

  __device__ TreeWalk(const AttendParams& p, const TreeList& list, int plen, int slot)
      : p(p), list(list), plen(plen), ptiles(key_tiles(plen)), slot(slot), at(list.at[slot]), end(list.end[slot]), b(-1) {}
  __device__ bool next() {
    if (at >= end) return false;
    kt0 = 0;
    if (b < 0) {
      b = list.b[slot];
      e = list.e[slot];
      const int3 x = tree_place(at - static_cast<int64_t>(list.cum[slot]) * p.s.heads, e.tiles, e.blocks);
      h = x.x;
      blk = x.y;
      kt0 = x.z;
    } else if (++blk == e.blocks) {
      blk = 0;
      if (++h == p.s.heads) {  // (an entry with tiles follows: the share goes on)
        h = 0;
        int found;
        e = tree_next_entry(p, list, ptiles, b + 1, &found);
        b = found;
      }
    }
    kt1 = static_cast<int>(min(static_cast<int64_t>(e.tiles), kt0 + (end - at)));
    at += kt1 - kt0;
    two = (2 * blk + 1) * p.s.per_tile < e.nodes;
    return true;
  }
  __device__ int first_node(int t) const { return (2 * blk + t) * p.s.per_tile; }
  // first query entry of row tile t, and its valid rows
  __device__ int entry(int t) const { return b * p.t.T + first_node(t); }
  __device__ int rows(int t) const {
    return min(p.s.per_tile, e.nodes - first_node(two ? t : 0)) * p.s.group;
  }
  __device__ bool whole() const { return kt0 == 0 && kt1 == e.tiles; }
  // where a unit that several workers have leaves its part: a worker has two such at most, its first and last
  __device__ int piece() const { return 2 * list.worker[slot] + (kt0 == 0); }
  // tokens from tile kt on
  __device__ int valid(int kt) const {
    return kt < ptiles ? plen - kt * TILE_KEYS : e.len - (kt - ptiles) * TILE_KEYS;
  }
  // first draft's place from tile kt's first key on
  __device__ int drafts(int kt) const {
    return kt < ptiles ? TILE_KEYS : e.len - e.nodes - (kt - ptiles) * TILE_KEYS;
  }
};

// The walk's tiles one by one.
struct TreeCursor {
  TreeWalk w;
  int u, u1, kt, seq, len, h;
  __device__ explicit TreeCursor(const TreeWalk& walk) : w(walk), u(-1), u1(0) {}
  __device__ bool step() {
    if (++u >= u1) {
      if (!w.next()) return false;
      u = w.kt0;
      u1 = w.kt1;
      h = w.h;
    }
    const bool shared = u < w.ptiles;
    kt = shared ? u : u - w.ptiles;
    seq = shared ? w.p.a.prefix : w.e.seq;
    len = shared ? w.plen : w.e.len;
    return true;
  }
};

// The tiles of two walks in turn. The first has as many as the second, or one more.
struct TreePairCursor {
  TreeCursor a, b;
  uint32_t n;
  int kt, seq, len, h;
  __device__ TreePairCursor(const TreeWalk& x, const TreeWalk& y) : a(x), b(y), n(0) {}
  __device__ bool step() {
    TreeCursor& c = n++ & 1 ? b : a;
    if (!c.step()) return false;
    kt = c.kt;
    seq = c.seq;
    len = c.len;
    h = c.h;
    return true;
  }
};

// The tiles of two walks in turn with what begins and ends with each: half t's unit (its how many-th) at
// its first and last tile.
struct TreePairUnits {
  TreeWalk a, b;
  int left[2], units[2];
  uint32_t n;
  int t, unit;
  bool first, last;
  __device__ TreePairUnits(const TreeWalk& x, const TreeWalk& y) : a(x), b(y), left{0, 0}, units{0, 0}, n(0) {}
  __device__ TreeWalk& walk() { return t ? b : a; }
  __device__ bool step() {
    t = n++ & 1;
    int x = left[t];
    first = x == 0;
    if (first) {
      TreeWalk& w = walk();
      if (!w.next()) return false;
      x = w.kt1 - w.kt0;
    }
    left[t] = --x;
    last = x == 0;
    unit = units[t];
    if (last) units[t] = unit + 1;
    return true;
  }
};

// The nodes that node `t` attends to, by a whole warp (each lane its own t; t >= nodes: none). A parent
// that is no earlier node is reported and counts as none.
static __device__ __noinline__ uint64_t tree_branch(const AttendParams& p, int b, int nodes, int t) {
  if (!p.t.parent) return t < nodes ? (uint64_t{2} << t) - 1 : 0;
  const int lane = threadIdx.x & 31;
  const int32_t* up = p.t.parent + static_cast<size_t>(b) * p.t.T;
  const int lo = lane < nodes ? up[lane] : -1, hi = lane + 32 < nodes ? up[lane + 32] : -1;
  uint64_t m = 0;
  bool go = t < nodes;
  int cur = go ? t : 0;
  while (__any_sync(0xffffffffu, go)) {
    const int x = __shfl_sync(0xffffffffu, lo, cur & 31), y = __shfl_sync(0xffffffffu, hi, cur & 31);
    if (go) {
      m |= uint64_t{1} << cur;
      const int next = cur < 32 ? x : y;
      if (next < -1 || next >= cur) atomicOr(p.a.v.err, kErrBadList);
      go = next >= 0 && next < cur;
      if (go) cur = next;
    }
  }
  return m;
}

// Which of the 64 keys from `drafts` places before the first draft on (behind it: negative) a node attends to.
__device__ __forceinline__ uint64_t tree_allowed(uint64_t branch, int drafts) {
  if (drafts >= 64) return ~uint64_t{0};
  if (drafts >= 0) return drafts ? ((uint64_t{1} << drafts) - 1) | branch << drafts : branch;
  return drafts > -64 ? branch >> -drafts : 0;
}

}  // namespace h2o
#endif  // __CUDACC__
