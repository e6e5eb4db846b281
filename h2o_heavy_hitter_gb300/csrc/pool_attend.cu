// Attention of single tokens over the paged cache on the tensor cores: a prefix
// that the whole batch shares, then each sequence's own tokens. For row (b,
// query head) with key head h: s_j = q . k_j / sqrt(d), lse = log sum_j
// exp(s_j), p_j = exp(s_j - lse), out = sum_j p_j v_j; scores grow by p.
//
// Bound: every stored key and value is read from HBM once, 4 d bytes a token and
// head, against 4 d flops per query row that sees it; below some 250 rows a head
// the bytes decide. So the design streams pages at full rate and keeps the rest
// out of the way:
//
// pool_attend_kernel. The work is one list of 128-key tiles, first those of the
//   prefix (one unit of tiles per key head and block of query rows: the queries
//   of all sequences are the rows of one matrix), then those of the sequences (a
//   unit per sequence and key head, whose rows are the head's query group). One
//   persistent CTA per SM takes an equal contiguous share of the list, whatever
//   the lengths are: they are read on the device, and every CTA finds its share
//   with one scan. A CTA's part of a unit gives an unnormalised output, a
//   maximum and a sum per row ("piece"); piece u + c is unique to unit u and CTA
//   c, as both only grow along the list.
//   TMA fetches the pages' boxes of page-size rows (two warps, K and V), one
//   thread issues S = Q K^T and O += P V (tcgen05, accumulators in TMEM), eight
//   warps do the softmax with a thread per row. With up to 128 rows the four
//   warps of half t take keys 64 t .. 64 t + 63 of every tile and their own
//   accumulator, so that two short softmax chains run side by side and no
//   maximum is exchanged; S is double-buffered, so the next tile's product is
//   ready when the softmax comes to it. With more rows the halves take a tile
//   of 128 rows each and share the K and V tiles. P is rounded to bf16, the
//   operand type of the second product; sums and logits stay in fp32.
//   What lies behind a sequence's end in its last page is not trusted: its
//   logits are replaced by -inf and its values in shared memory by zeros.
// pool_finish_kernel joins the pieces of each row in fixed order and adds the
//   probabilities to the sequences' scores, from the logits that the first
//   kernel left (4 bytes per key and row, against 4 d of keys and values).
// pool_prefix_score_kernel adds the prefix's: S^T = K Q^T again, with one thread
//   per key, p = 2^(s - lse) summed over all rows in order. Recomputing reads K
//   once more (2 d bytes a key) where keeping the logits of all rows would move 8
//   bytes a key and row.
#include <algorithm>

#include "common.cuh"
#include "device_state.h"
#include "kernels.h"
#include "pool.h"
#include "scan.cuh"
#include "tc.cuh"

namespace h2o {
namespace {

constexpr int TILE_KEYS = 128;
constexpr int TILE_ROWS = 128;

// ------------------------------------------------------------------ the work list
// Host-computed shape of a call.
struct Shape {
  int n, heads, group, d;
  int per_tile;  // sequences whose query groups share a tile of rows: 128 / group
  int nq;        // row tiles per head
  int blocks;    // blocks of two row tiles per head (0 without a prefix)
  int grid;      // CTAs of the attention kernel
};

Shape shape_of(const AttendArgs& a, int sms) {
  Shape s{};
  s.n = a.n;
  s.heads = a.v.heads;
  s.group = a.group;
  s.d = a.v.d;
  s.per_tile = TILE_ROWS / a.group;
  s.nq = (a.n + s.per_tile - 1) / s.per_tile;
  s.blocks = a.prefix >= 0 ? (s.nq + 1) / 2 : 0;
  s.grid = sms;
  return s;
}

// Scratch of a call, in order.
struct Scratch {
  int* seq;       // [n] sequence of a row, -1 skipped
  int* cum;       // [n + 1] 128-key tiles of the sequences before
  float* nlse;    // [heads][nq][128] -lse (base 2) of a prefix row, -inf: not counted
  float2* pml;    // prefix pieces [heads * blocks + grid][2][128] {max, sum}
  float2* tml;    // own pieces [n * heads + grid][group] {max, sum}
  float* po;      // prefix pieces' outputs [..][d]
  float* to;      // own pieces' outputs [..][d]
  float* logits;  // [n][heads][group][cap] base-2 logits (accumulate only)
};

size_t scratch_layout(const Shape& s, int cap, bool accumulate, void* base, Scratch* out) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = static_cast<char*>(base) + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const size_t pp = s.blocks ? static_cast<size_t>(s.heads) * s.blocks + s.grid : 0;
  const size_t tp = static_cast<size_t>(s.n) * s.heads + s.grid;
  Scratch w{};
  w.seq = reinterpret_cast<int*>(take(s.n * sizeof(int)));
  w.cum = reinterpret_cast<int*>(take((s.n + 1) * sizeof(int)));
  w.nlse = reinterpret_cast<float*>(take(s.blocks ? static_cast<size_t>(s.heads) * s.nq * 512 : 0));
  w.pml = reinterpret_cast<float2*>(take(pp * 256 * sizeof(float2)));
  w.tml = reinterpret_cast<float2*>(take(tp * s.group * sizeof(float2)));
  w.po = reinterpret_cast<float*>(take(pp * 256 * s.d * sizeof(float)));
  w.to = reinterpret_cast<float*>(take(tp * s.group * s.d * sizeof(float)));
  w.logits = reinterpret_cast<float*>(
      take(accumulate ? static_cast<size_t>(s.n) * s.heads * s.group * cap * sizeof(float) : 0));
  if (out) *out = w;
  return at;
}

struct Params {
  AttendArgs a;
  Shape s;
  Scratch w;
  float qscale;  // log2(e) / sqrt(d)
};

// A sequence's length, -1 (reported when `report`) for a state that no call leaves.
__device__ __forceinline__ int checked_length(const PoolView& v, int seq, bool report) {
  const int len = v.meta[2 * seq];
  if (len >= 0 && len <= v.cap) return len;
  if (report) atomicOr(v.err, kErrBadState);
  return -1;
}

// CTAs that get a share of `total` tiles: none is left without one between two that have.
__device__ __forceinline__ int64_t sharers(int64_t total, int grid) {
  return min(total, static_cast<int64_t>(grid));
}

__device__ __forceinline__ int key_tiles(int len) { return (len + TILE_KEYS - 1) / TILE_KEYS; }

// The list in shared memory, and a walk along one CTA's share of it.
struct List {
  int seq[kPoolMaxList];
  int len[kPoolMaxList];
  int cum[kPoolMaxList + 2];  // one more than used, for the alignment of what follows
};

struct Walk {
  const Params& p;
  const List& list;
  int ptiles, plen;      // tiles and tokens of the prefix
  int64_t ptotal;        // tiles of all prefix units
  int64_t at, end;
  // the unit: its head, its row block (prefix) or list entry, its tiles in this share
  bool prefix, two;
  int h, b, seq, len, kt0, kt1, piece;

  __device__ Walk(const Params& p, const List& list, int plen, int cta)
      : p(p), list(list), plen(plen) {
    ptiles = key_tiles(plen);
    ptotal = static_cast<int64_t>(p.s.heads) * p.s.blocks * ptiles;
    const int64_t total = ptotal + static_cast<int64_t>(list.cum[p.s.n]) * p.s.heads;
    const int64_t ctas = sharers(total, p.s.grid);
    at = cta < ctas ? total * cta / ctas : total;
    end = cta < ctas ? total * (cta + 1) / ctas : total;
    piece = cta;
  }
  __device__ int rows(int t) const {  // valid rows of the unit's row tile t
    if (!prefix) return p.s.group;
    const int first = (2 * b + (two ? t : 0)) * p.s.per_tile;
    return min(p.s.per_tile, p.s.n - first) * p.s.group;
  }
  __device__ bool next(int cta) {
    if (at >= end) return false;
    int tiles;
    prefix = at < ptotal;
    if (prefix) {
      const int u = static_cast<int>(at / ptiles);
      kt0 = static_cast<int>(at - static_cast<int64_t>(u) * ptiles);
      h = u / p.s.blocks;
      b = u - h * p.s.blocks;
      two = 2 * b + 1 < p.s.nq;
      seq = p.a.prefix;
      len = plen;
      tiles = ptiles;
      piece = u + cta;
    } else {
      const int64_t q = at - ptotal;
      int lo = 0, hi = p.s.n - 1;  // the last entry that begins at or before q and has tiles
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (static_cast<int64_t>(list.cum[mid]) * p.s.heads <= q)
          lo = mid;
        else
          hi = mid - 1;
      }
      b = lo;
      tiles = list.cum[b + 1] - list.cum[b];
      const int r = static_cast<int>(q - static_cast<int64_t>(list.cum[b]) * p.s.heads);
      h = r / tiles;
      kt0 = r - h * tiles;
      two = false;
      seq = list.seq[b];
      len = list.len[b];
      piece = b * p.s.heads + h + cta;
    }
    kt1 = static_cast<int>(min(static_cast<int64_t>(tiles), kt0 + (end - at)));
    at += kt1 - kt0;
    return true;
  }
};

// Fills the list: skipped and refused entries have seq -1 and no tiles. An entry
// is refused for an index outside the pool, the prefix's, or one named before;
// repeats are looked for one by one only where a hashed bit says that there may
// be some. Blockwide; `bits`: 4 KB; `report`: this block sets the error word.
__device__ void build_list(const AttendArgs& a, List& list, uint32_t* bits, int* wsum,
                           bool report) {
  const PoolView& v = a.v;
  const int tid = threadIdx.x, nt = blockDim.x, n = a.n;
  for (int i = tid; i < 1024; i += nt) bits[i] = 0;
  __syncthreads();
  bool seen = false;
  for (int b = tid; b < n; b += nt) {
    int s = a.seqs[b];
    if (s != -1 && (s < 0 || s >= v.seqs || s == a.prefix)) {
      if (report) atomicOr(v.err, kErrBadList);
      s = -1;
    }
    list.seq[b] = s;
    list.len[b] = s >= 0 ? checked_length(v, s, report) : -1;
    if (s >= 0) seen |= (atomicOr(&bits[(s >> 5) & 1023], 1u << (s & 31)) >> (s & 31)) & 1u;
  }
  if (__syncthreads_or(seen)) {
    for (int b = tid; b < n; b += nt) {
      const int s = a.seqs[b];
      if (s < 0) continue;
      for (int j = 0; j < b; ++j)
        if (a.seqs[j] == s) {
          if (report) atomicOr(v.err, kErrBadList);
          list.len[b] = -1;
          break;
        }
    }
  }
  __syncthreads();
  const int per = (n + nt - 1) / nt, b0 = min(n, tid * per), b1 = min(n, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    if (list.len[b] < 0) list.seq[b] = -1;
    mine += key_tiles(max(0, list.len[b]));
  }
  int total;
  int at = block_exclusive_scan(mine, wsum, &total);
  for (int b = b0; b < b1; ++b) {
    list.cum[b] = at;
    at += key_tiles(max(0, list.len[b]));
  }
  if (tid == 0) list.cum[n] = total;
  __syncthreads();
}

// ------------------------------------------------------------------ attention
constexpr int kWarpK = 0;        // TMA loads of Q and K
constexpr int kWarpMMA = 1;      // owns TMEM, issues every tcgen05.mma
constexpr int kWarpV = 2;        // TMA loads of V
constexpr int kWarpSoftmax = 3;  // warps 3..6: half or row tile 0, 7..10: 1
constexpr int kThreads = 11 * 32;

template <int D>
struct Cfg {
  static constexpr int ST = D == 128 ? 2 : 4;  // K and V tiles in flight, each
  static constexpr int TILE = TILE_KEYS * D * 2;
  static constexpr uint32_t O_COL = 256;  // S buffers at columns 0 and 128, O of half t at 256 + 128 t
  static constexpr int MERGE = 32 * (D + 2) * 4;
  static constexpr size_t SMEM =
      static_cast<size_t>(2 + 2 * ST) * TILE + MERGE + sizeof(List) + 1024 + 1024;
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[4], k_empty[4];
  uint64_t v_full[4], v_empty[4];
  uint64_t s_full[2], p_ready[2];  // by S buffer
  uint64_t pv_done[2];             // by S buffer
  uint64_t o_last[2], o_free[2];   // one phase per unit
  uint64_t m_full, m_empty;        // merge buffer, one phase per own-token unit
  uint32_t tmem;
  int wsum[33];
};
static_assert(sizeof(Bars) <= 1024, "Bars must fit the space reserved in Cfg::SMEM");

// One warp fetches a 128-key tile of a sequence's page list: lane i the boxes of
// page i of the tile, those behind the last token left out. `page` is the lane's
// table entry (fetch_page), loaded before the wait for the stage.
__device__ __forceinline__ int fetch_page(const PoolView& v, int seq, int len, int kt, int lane) {
  const int per = TILE_KEYS >> v.shift, j = kt * per + lane;
  if (lane >= per || j << v.shift >= len) return -1;
  int p = v.table[static_cast<size_t>(seq) * v.width + j];
  if (p < 0 || p >= v.pages) {  // reported; some page of the pool is read in its place
    atomicOr(v.err, kErrBadState);
    p = 0;
  }
  return p;
}

template <int D>
__device__ __forceinline__ void fetch_tile(const PoolView& v, const CUtensorMap* map, uint8_t* dst,
                                           int page, int head, int len, int kt, int lane,
                                           uint64_t* bar) {
  const int left = len - kt * TILE_KEYS, per = TILE_KEYS >> v.shift;
  const int boxes = min(per, (left + v.page - 1) >> v.shift);
  if (lane == 0) mbar_arrive_expect_tx(bar, boxes * v.page * D * 2);
  __syncwarp();
  if (page < 0) return;
  const int row = (page * v.heads + head) << v.shift;
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
    tma_load_2d(dst + c * kBoxBytes + (lane << v.shift) * 128, map, c * 64, row, bar);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    pool_attend_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap t1,
                       const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ Params p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + 2 * C::TILE;
  uint8_t* sV = sK + C::ST * C::TILE;
  float* merge = reinterpret_cast<float*>(sV + C::ST * C::TILE);
  List& list = *reinterpret_cast<List*>(reinterpret_cast<uint8_t*>(merge) + C::MERGE);
  Bars* bars = reinterpret_cast<Bars*>(&list + 1);
  const PoolView& v = p.a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_ready[i], 8);
      mbar_init(&bars->pv_done[i], 1);
      mbar_init(&bars->o_last[i], 1);
      mbar_init(&bars->o_free[i], 4);
    }
    for (int i = 0; i < C::ST; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 1);
      mbar_init(&bars->v_full[i], 1);
      mbar_init(&bars->v_empty[i], 1);
    }
    mbar_init(&bars->m_full, 1);
    mbar_init(&bars->m_empty, 1);
    fence_barrier_init();
  }
  if (warp == kWarpMMA) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  if (warp == kWarpK && lane == 0) {
    tma_prefetch_map(&tq);
    tma_prefetch_map(&t1);
    tma_prefetch_map(&tk);
  }
  if (warp == kWarpV && lane == 0) tma_prefetch_map(&tv);
  build_list(p.a, list, reinterpret_cast<uint32_t*>(merge), bars->wsum, cta == 0);
  const int plen = p.a.prefix >= 0 ? max(0, checked_length(v, p.a.prefix, threadIdx.x == 0)) : 0;
  if (cta == 0) {
    for (int i = threadIdx.x; i < p.s.n; i += kThreads) p.w.seq[i] = list.seq[i];
    for (int i = threadIdx.x; i <= p.s.n; i += kThreads) p.w.cum[i] = list.cum[i];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  Walk w(p, list, plen, cta);

  if (warp == kWarpK || warp == kWarpV) {
    // ---------------------------------------------------------------- TMA loads
    const bool is_k = warp == kWarpK;
    uint64_t* full = is_k ? bars->k_full : bars->v_full;
    uint64_t* empty = is_k ? bars->k_empty : bars->v_empty;
    uint8_t* ring = is_k ? sK : sV;
    const CUtensorMap* map = is_k ? &tk : &tv;
    uint32_t g = 0, qn = 0;
    bool ok = true;
    while (ok && w.next(cta)) {
      for (int t = 0; is_k && ok && t < (w.two ? 2 : 1); ++t, ++qn) {
        const uint32_t qb = qn & 1;
        if (qn >= 2 && !warp_wait(&bars->q_empty[qb], ((qn >> 1) - 1) & 1, v.err)) ok = false;
        if (!ok || lane) continue;
        const CUtensorMap* qm = w.prefix ? &tq : &t1;
        const int entry = w.prefix ? (2 * w.b + t) * p.s.per_tile : w.b;
        const int entries = w.prefix ? p.s.per_tile : 1;
        mbar_arrive_expect_tx(&bars->q_full[qb], entries * p.s.group * D * 2);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(sQ + qb * C::TILE + c * kBoxBytes, qm, c * 64, 0, w.h, entry,
                      &bars->q_full[qb]);
      }
      for (int kt = w.kt0; ok && kt < w.kt1; ++kt, ++g) {
        const int page = fetch_page(v, w.seq, w.len, kt, lane);
        const uint32_t st = g % C::ST;
        if (g >= C::ST && !warp_wait(&empty[st], ((g / C::ST) - 1) & 1, v.err)) {
          ok = false;
          break;
        }
        fetch_tile<D>(v, map, ring + st * C::TILE, page, w.h, w.len, kt, lane, &full[st]);
      }
    }
  } else if (warp == kWarpMMA) {
    // ---------------------------------------------------------------- MMA issuer
    // S j is followed by the P V of S j - 1, so the softmax of one S overlaps the
    // product of the next; the S buffer of j is that of j - 2, whose P V is issued.
    if (lane == 0) {
      constexpr uint32_t idesc_qk = idesc_bf16(TILE_ROWS, TILE_KEYS, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16(TILE_ROWS, D, 0, 1);
      const uint64_t dq0 = desc_kmajor<D>(sQ, 0), dk0 = desc_kmajor<D>(sK, 0);
      const uint64_t dv0 = smem_desc(sV, kBoxBytes, 1024);
      uint32_t g = 0, qn = 0, j = 0;
      int e = 0;
      bool ok = true;
      struct {
        bool live = false, two, first, last, frees;
        int t, e;
        uint32_t j, g;
      } pv;
      auto issue_pv = [&]() -> bool {
        const uint32_t st = pv.g % C::ST, buf = pv.j & 1;
        if (!mbar_wait(&bars->p_ready[buf], (pv.j >> 1) & 1, v.err) ||
            !mbar_wait(&bars->v_full[st], (pv.g / C::ST) & 1, v.err))
          return false;
        if (pv.first && pv.e > 0) {
          for (int t = 0; t < 2; ++t)
            if ((!pv.two || t == pv.t) && !mbar_wait(&bars->o_free[t], (pv.e - 1) & 1, v.err))
              return false;
        }
        tc_fence_after();
        const uint64_t vb = dv0 + static_cast<uint64_t>(st * (C::TILE >> 4));
        const uint32_t s_tm = tmem + buf * 128;
        // B = V tile, MN-major: 16 keys = two 8-row swizzle atoms (2048 bytes)
#pragma unroll
        for (int kk = 0; kk < TILE_KEYS / 16; ++kk) {
          const int half = kk >> 2;
          const uint32_t o = tmem + C::O_COL + (pv.two ? pv.t : half) * 128;
          const uint32_t a = s_tm + (pv.two ? kk * 8 : half * 64 + (kk & 3) * 8);
          const bool fresh = pv.first && (pv.two ? kk == 0 : (kk & 3) == 0);
          umma_ts(o, a, vb + kk * (2048 >> 4), idesc_pv, fresh ? 0u : 1u);
        }
        umma_commit(&bars->pv_done[buf]);
        if (pv.frees) umma_commit(&bars->v_empty[st]);
        if (pv.last)
          for (int t = 0; t < 2; ++t)
            if (!pv.two || t == pv.t) umma_commit(&bars->o_last[t]);
        return true;
      };
      while (ok && w.next(cta)) {
        const int nt = w.two ? 2 : 1;
        for (int kt = w.kt0; ok && kt < w.kt1; ++kt, ++g) {
          const uint32_t st = g % C::ST;
          for (int t = 0; ok && t < nt; ++t, ++j) {
            const uint32_t qb = (qn + t) & 1;
            if ((kt == w.kt0 && !mbar_wait(&bars->q_full[qb], ((qn + t) >> 1) & 1, v.err)) ||
                (t == 0 && !mbar_wait(&bars->k_full[st], (g / C::ST) & 1, v.err))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t kb = dk0 + static_cast<uint64_t>(st * (C::TILE >> 4));
            const uint64_t qd = dq0 + static_cast<uint64_t>(qb * (C::TILE >> 4));
            const uint32_t d_tm = tmem + (j & 1) * 128;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = ((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4;
              umma_ss(d_tm, qd + off, kb + off, idesc_qk, kk > 0);
            }
            umma_commit(&bars->s_full[j & 1]);
            if (t == nt - 1) umma_commit(&bars->k_empty[st]);
            if (kt == w.kt1 - 1) umma_commit(&bars->q_empty[qb]);
            if (pv.live && !issue_pv()) {
              ok = false;
              break;
            }
            pv.live = true;
            pv.two = w.two;
            pv.first = kt == w.kt0;
            pv.last = kt == w.kt1 - 1;
            pv.frees = t == nt - 1;
            pv.t = t;
            pv.e = e;
            pv.j = j;
            pv.g = g;
          }
        }
        qn += nt;
        ++e;
      }
      if (ok && pv.live) issue_pv();
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int t = (warp - kWarpSoftmax) >> 2, quad = warp & 3;
    const int r = quad * 32 + lane, tid = ((warp - kWarpSoftmax) & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t o_tm = tmem + lane_off + C::O_COL + t * 128;
    uint32_t j0 = 0, g = 0;
    int e = 0, tails = 0;
    bool ok = true;
    while (ok && w.next(cta)) {
      const int rows = w.rows(t), step = w.two ? 2 : 1;
      const bool active = quad * 32 < rows;  // warp-uniform
      const int chunks = w.two ? 2 : 1, col0 = w.two ? 0 : 64 * t;
      float m = -INFINITY, l = 0.f;
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++g) {
        const uint32_t jj = j0 + (kt - w.kt0) * step, j = w.two ? jj + t : jj;
        const uint32_t s_tm = tmem + lane_off + (j & 1) * 128;
        if (!warp_wait(&bars->s_full[j & 1], (j >> 1) & 1, v.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int valid = w.len - kt * TILE_KEYS;  // may exceed 128
        if (active) {
          uint32_t s[64];
          float mx = -INFINITY;
          for (int c = 0; c < chunks; ++c) {
            const int first = col0 + 64 * c;
            tmem_ld32(s_tm + first, s);
            tmem_ld32(s_tm + first + 32, s + 32);
            tmem_wait_ld();
            if (first + 64 > valid) {
#pragma unroll
              for (int x = 0; x < 64; ++x)
                if (first + x >= valid) s[x] = __float_as_uint(-INFINITY);
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < 64; x += 8)
#pragma unroll
              for (int y = 0; y < 4; ++y)
                m4[y] = fmax3(m4[y], __uint_as_float(s[x + y]), __uint_as_float(s[x + 4 + y]));
            mx = fmax3(fmax3(mx, m4[0], m4[1]), m4[2], m4[3]);
          }
          mx *= p.qscale;
          float alpha = 1.f;
          bool rescale = false;
          if (mx > m + 8.f) {
            rescale = kt > w.kt0 && l > 0.f;
            if (rescale) alpha = ex2(m - mx);
            m = mx;
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const uint64_t sc2 = f2_pack(p.qscale, p.qscale), nm2 = f2_pack(-ref, -ref);
          uint64_t rs2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
          const bool keep = p.w.logits && !w.prefix && r < rows;
          for (int c = 0; c < chunks; ++c) {
            const int first = col0 + 64 * c;
            if (chunks > 1) {
              tmem_ld32(s_tm + first, s);
              tmem_ld32(s_tm + first + 32, s + 32);
              tmem_wait_ld();
              if (first + 64 > valid) {
#pragma unroll
                for (int x = 0; x < 64; ++x)
                  if (first + x >= valid) s[x] = __float_as_uint(-INFINITY);
              }
            }
            if (keep) {
              float4* dst = reinterpret_cast<float4*>(
                  p.w.logits +
                  ((static_cast<size_t>(w.b) * p.s.heads + w.h) * p.s.group + r) * v.cap +
                  kt * TILE_KEYS + first);
              // a page of at least 16 tokens ends the row at a multiple of 16
#pragma unroll
              for (int x = 0; x < 16; ++x)
                if (first + 4 * x < valid)
                  dst[x] = make_float4(__uint_as_float(s[4 * x]) * p.qscale,
                                       __uint_as_float(s[4 * x + 1]) * p.qscale,
                                       __uint_as_float(s[4 * x + 2]) * p.qscale,
                                       __uint_as_float(s[4 * x + 3]) * p.qscale);
            }
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              uint32_t pk[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                float a, b;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[cc * 16 + 2 * x]),
                                         __uint_as_float(s[cc * 16 + 2 * x + 1])),
                                 sc2, nm2),
                          a, b);
                const float p0 = ex2(a), p1 = ex2(b);
                rs2[x & 1] = f2_add(rs2[x & 1], f2_pack(p0, p1));
                pk[x] = pack_bf16x2(p0, p1);
              }
              // P over S columns already read: this half's, or (two chunks) the first 64
              tmem_st8(s_tm + (w.two ? 32 * c : col0) + cc * 8, pk);
            }
          }
          float r0, r1, r2, r3;
          f2_unpack(rs2[0], r0, r1);
          f2_unpack(rs2[1], r2, r3);
          l = fmaf(l, alpha, (r0 + r1) + (r2 + r3));
          // the whole warp rescales its O rows when any of its rows raised the max;
          // the P V before this S must have completed (with two row tiles it has:
          // it was issued before this S)
          if (__any_sync(0xffffffffu, rescale)) {
            // (on its own barrier, whose phase before belongs to the P V of j - 3: a
            // parity wait may be one phase behind or level, never two)
            if (!w.two && !warp_wait(&bars->pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, v.err)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(o_tm + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
              tmem_st32(o_tm + c * 32, o);
            }
          }
        }
        if (valid < TILE_KEYS) {  // values behind the end count as zero, whatever they are
          const uint32_t st = g % C::ST;
          if (!warp_wait(&bars->v_full[st], (g / C::ST) & 1, v.err)) {
            ok = false;
            break;
          }
          const int lo = w.two ? 0 : 64 * t, hi = w.two ? TILE_KEYS : lo + 64;
          const int from = max(lo, valid);
          for (int x = tid; x < (hi - from) * (D / 8); x += 128) {
            const int row = from + x / (D / 8), c = x % (D / 8);
            *reinterpret_cast<uint4*>(sV + st * C::TILE + (c >> 3) * kBoxBytes + row * 128 +
                                      (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_n(&bars->p_ready[j & 1], w.two ? 2 : 1);
      }
      if (!ok) break;
      // ---- the piece: O out of TMEM, which the next unit may then use
      if (!warp_wait(&bars->o_last[t], e & 1, v.err)) break;
      tc_fence_after();
      const bool merges = !w.prefix;  // rows of own tokens: at most 32, both halves in quadrant 0
      if (active) {
        if (merges && t == 1) {
          if (tails > 0 && !warp_wait(&bars->m_empty, (tails - 1) & 1, v.err)) break;
        } else if (merges) {
          if (!warp_wait(&bars->m_full, tails & 1, v.err)) break;
        }
        float wa = 1.f, wb = 0.f;
        if (merges && t == 0) {
          const float mb = merge[D * 32 + lane], lb = merge[(D + 1) * 32 + lane];
          const float top = fmaxf(m, mb);
          wa = m == -INFINITY ? 0.f : ex2(m - top);
          wb = mb == -INFINITY ? 0.f : ex2(mb - top);
          l = l * wa + lb * wb;
          m = top;
        }
        const size_t rec = w.prefix ? (static_cast<size_t>(w.piece) * 2 + t) * TILE_ROWS + r
                                    : static_cast<size_t>(w.piece) * p.s.group + r;
        float* po = (w.prefix ? p.w.po : p.w.to) + rec * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_tm + c * 32, o);
          tmem_wait_ld();
          if (merges && t == 1) {
#pragma unroll
            for (int x = 0; x < 32; ++x) merge[(c * 32 + x) * 32 + lane] = __uint_as_float(o[x]);
          } else if (r < rows) {
            if (merges) {
#pragma unroll
              for (int x = 0; x < 32; ++x)
                o[x] = __float_as_uint(__uint_as_float(o[x]) * wa +
                                       merge[(c * 32 + x) * 32 + lane] * wb);
            }
#pragma unroll
            for (int x = 0; x < 8; ++x)
              reinterpret_cast<uint4*>(po + c * 32)[x] =
                  make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
        }
        if (merges && t == 1) {
          merge[D * 32 + lane] = m;
          merge[(D + 1) * 32 + lane] = l;
        } else if (r < rows) {
          (w.prefix ? p.w.pml : p.w.tml)[rec] = make_float2(m, l);
        }
        __syncwarp();
        if (merges && lane == 0) mbar_arrive(t ? &bars->m_full : &bars->m_empty);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_free[t]);
      tails += merges;
      j0 += (w.kt1 - w.kt0) * step;
      ++e;
    }
  }
  grid_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ joining the pieces
constexpr int kFinishThreads = 128;

// CTA of the attention kernel whose share holds tile `at` of `total`.
__device__ __forceinline__ int owner(int64_t at, int64_t total, int grid) {
  return static_cast<int>(((at + 1) * sharers(total, grid) - 1) / total);
}

// Block (b, key head; chunk of keys). A warp joins a row: its prefix pieces, then
// its own. All chunks need the row's lse for the scores, the first writes it.
template <int D>
__global__ void __launch_bounds__(kFinishThreads)
    pool_finish_kernel(const __grid_constant__ Params p) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ float s_lse[kPoolMaxGroup];
  const PoolView& v = p.a.v;
  const int b = blockIdx.x / p.s.heads, h = blockIdx.x % p.s.heads, group = p.s.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seq = p.w.seq[b];
  const int qt = b / p.s.per_tile, r0 = (b - qt * p.s.per_tile) * group;
  float* nlse = p.w.nlse + (static_cast<size_t>(h) * p.s.nq + qt) * TILE_ROWS + r0;
  if (seq < 0) {
    if (p.s.blocks && blockIdx.y == 0)
      for (int g = threadIdx.x; g < group; g += kFinishThreads) nlse[g] = -INFINITY;
    return;
  }
  const int plen = p.a.prefix >= 0 ? max(0, checked_length(v, p.a.prefix, false)) : 0;
  const int ptiles = key_tiles(plen), len = v.meta[2 * seq];
  const int64_t ptotal = static_cast<int64_t>(p.s.heads) * p.s.blocks * ptiles;
  const int64_t total = ptotal + static_cast<int64_t>(p.w.cum[p.s.n]) * p.s.heads;
  // pieces [pa, pa + np) of the prefix unit, each of one or two records; [ta, ta + nt) of the own
  int np = 0, nt = 0, pa = 0, ta = 0, recs = 1, rec0 = 0;
  if (ptiles) {
    const int u = h * p.s.blocks + (qt >> 1);
    const int64_t at = static_cast<int64_t>(u) * ptiles;
    const int c0 = owner(at, total, p.s.grid);
    np = owner(at + ptiles - 1, total, p.s.grid) - c0 + 1;
    pa = u + c0;
    if ((qt | 1) < p.s.nq)
      rec0 = qt & 1;  // a block of two row tiles: a record per tile
    else
      recs = 2;       // one row tile: a record per half of the keys
  }
  const int tiles = p.w.cum[b + 1] - p.w.cum[b];
  if (tiles) {
    const int64_t at = ptotal + static_cast<int64_t>(p.w.cum[b]) * p.s.heads + static_cast<int64_t>(h) * tiles;
    const int c0 = owner(at, total, p.s.grid);
    nt = owner(at + tiles - 1, total, p.s.grid) - c0 + 1;
    ta = b * p.s.heads + h + c0;
  }
  const int prs = np * recs, all = prs + nt;
  for (int g = warp; g < group; g += kFinishThreads / 32) {
    auto rec = [&](int i) -> size_t {  // row of record i in its array
      if (i < prs)
        return (static_cast<size_t>(pa + i / recs) * 2 + rec0 + i % recs) * TILE_ROWS + r0 + g;
      return static_cast<size_t>(ta + i - prs) * group + g;
    };
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < all; i += 32) {
      const float2 x = (i < prs ? p.w.pml : p.w.tml)[rec(i)];
      const float top = fmaxf(m, x.x);
      if (top != -INFINITY) {
        l = l * ex2(m - top) + x.y * ex2(x.x - top);
        m = top;
      } else {
        l += x.y;  // a NaN sum stays one
      }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m, off), lo = __shfl_xor_sync(0xffffffffu, l, off);
      const float top = fmaxf(m, mo);
      if (top != -INFINITY) l = l * ex2(m - top) + lo * ex2(mo - top);
      else l += lo;
      m = top;
    }
    const float lse = __shfl_sync(0xffffffffu, all ? m + log2f(l) : -INFINITY, 0);
    if (lane == 0) s_lse[g] = lse;
    if (blockIdx.y) continue;
    float acc[D / 32] = {};
    for (int i = 0; i < all; ++i) {
      const size_t at = rec(i);
      const float wgt = ex2((i < prs ? p.w.pml : p.w.tml)[at].x - lse);
      const float* o = (i < prs ? p.w.po : p.w.to) + at * D + lane * (D / 32);
      if (wgt == 0.f) continue;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) acc[x] = fmaf(wgt, o[x], acc[x]);
    }
    const size_t row = (static_cast<size_t>(b) * p.s.heads + h) * group + g;
    uint32_t* out = static_cast<uint32_t*>(p.a.out) + row * (D / 2) + lane * (D / 64);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) out[x] = pack_bf16x2(acc[2 * x], acc[2 * x + 1]);
    if (lane == 0) {
      if (p.a.lse) p.a.lse[row] = lse * 0.69314718055994531f;  // ln 2
      if (p.s.blocks) nlse[g] = -lse;
    }
  }
  if (!p.w.logits) return;
  __syncthreads();
  const float* L = p.w.logits + (static_cast<size_t>(b) * p.s.heads + h) * group * v.cap;
  float* score = v.score + (static_cast<size_t>(seq) * v.heads + h) * v.cap;
  for (int j = blockIdx.y * kFinishThreads + threadIdx.x; j < len; j += gridDim.y * kFinishThreads) {
    float sum = 0.f;
    for (int g = 0; g < group; ++g) sum += ex2(L[static_cast<size_t>(g) * v.cap + j] - s_lse[g]);
    score[j] += sum;
  }
}

// ------------------------------------------------------------------ scores of the prefix
constexpr int kScoreThreads = 10 * 32;  // warps: 0 TMA, 1 MMA, 2..5 even key tiles, 6..9 odd ones

template <int D>
struct ScoreCfg {
  static constexpr int KST = D == 128 ? 4 : 8;
  static constexpr int TILE = TILE_KEYS * D * 2;
  static constexpr size_t SMEM = static_cast<size_t>(2 + KST) * TILE + 1024 + 512;
};

struct ScoreBars {
  uint64_t k_full[8], k_empty[8];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[4], s_free[4];  // S buffers 2 t + (0, 1) of half t
  uint32_t tmem;
};
static_assert(sizeof(ScoreBars) <= 512, "ScoreBars must fit the space reserved in ScoreCfg::SMEM");

// Persistent: a CTA takes an equal contiguous share of the (head, key tile)
// list. The row tiles of a head stay in shared memory when there are at most
// two; more are fetched again for every key tile. A fill is one load of a row
// tile: fill f lies in buffer f & 1.
template <int D>
__global__ void __launch_bounds__(kScoreThreads, 1)
    pool_prefix_score_kernel(const __grid_constant__ CUtensorMap tq,
                             const __grid_constant__ CUtensorMap tk, const __grid_constant__ Params p) {
  using C = ScoreCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + 2 * C::TILE;
  ScoreBars* bars = reinterpret_cast<ScoreBars*>(sK + C::KST * C::TILE);
  const PoolView& v = p.a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::KST; ++i) {
      mbar_init(&bars->k_full[i], 1);
      mbar_init(&bars->k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_free[i], 4);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tq);
    tma_prefetch_map(&tk);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  grid_dependency_wait();
  const int len = max(0, checked_length(v, p.a.prefix, false)), tiles = key_tiles(len);
  const int64_t total = static_cast<int64_t>(tiles) * p.s.heads;
  const int64_t begin = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;
  const int nq = p.s.nq, group = p.s.group;
  const bool stay = nq <= 2;

  if (warp == 0) {
    uint32_t g = 0, f = 0;
    bool ok = true;
    int last = -1;
    for (int64_t it = begin; ok && it < end; ++it, ++g) {
      const int h = static_cast<int>(it / tiles), kt = static_cast<int>(it - static_cast<int64_t>(h) * tiles);
      const int page = fetch_page(v, p.a.prefix, len, kt, lane);
      const uint32_t st = g % C::KST;
      if (g >= C::KST && !warp_wait(&bars->k_empty[st], ((g / C::KST) - 1) & 1, v.err)) break;
      fetch_tile<D>(v, &tk, sK + st * C::TILE, page, h, len, kt, lane, &bars->k_full[st]);
      if (stay && h == last) continue;
      last = h;
      for (int qt = 0; qt < nq; ++qt, ++f) {
        const uint32_t qb = f & 1;
        if (f >= 2 && !warp_wait(&bars->q_empty[qb], ((f >> 1) - 1) & 1, v.err)) {
          ok = false;
          break;
        }
        if (lane) continue;
        mbar_arrive_expect_tx(&bars->q_full[qb], p.s.per_tile * group * D * 2);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(sQ + qb * C::TILE + c * kBoxBytes, &tq, c * 64, 0, h, qt * p.s.per_tile,
                      &bars->q_full[qb]);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint64_t dq0 = desc_kmajor<D>(sQ, 0), dk0 = desc_kmajor<D>(sK, 0);
      uint32_t g = 0, f0 = 0, cnt[2] = {0, 0};  // f0: fill of the head's (or tile's) row tile 0
      bool ok = true;
      int last = -1;
      for (int64_t it = begin; ok && it < end; ++it, ++g) {
        const int h = static_cast<int>(it / tiles);
        const bool fresh = !stay || h != last;  // row tiles newly filled
        if (fresh && last >= 0) f0 += nq;
        last = h;
        // the row tiles' last use: with the head's last key tile of this share, or at once
        const bool done = !stay || it + 1 == end || static_cast<int>((it + 1) / tiles) != h;
        const uint32_t st = g % C::KST;
        const int t = g & 1;
        if (!mbar_wait(&bars->k_full[st], (g / C::KST) & 1, v.err)) break;
        for (int qt = 0; qt < nq; ++qt) {
          const uint32_t f = f0 + qt, qb = f & 1, buf = 2 * t + (cnt[t] & 1);
          if ((fresh && !mbar_wait(&bars->q_full[qb], (f >> 1) & 1, v.err)) ||
              (cnt[t] >= 2 && !mbar_wait(&bars->s_free[buf], ((cnt[t] >> 1) - 1) & 1, v.err))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int rows = min(p.s.per_tile, p.s.n - qt * p.s.per_tile) * group;
          const uint32_t idesc = idesc_bf16(TILE_KEYS, (rows + 15) / 16 * 16, 0, 0);
          const uint64_t kb = dk0 + static_cast<uint64_t>(st * (C::TILE >> 4));
          const uint64_t qd = dq0 + static_cast<uint64_t>(qb * (C::TILE >> 4));
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = ((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4;
            umma_ss(tmem + buf * 128, kb + off, qd + off, idesc, kk > 0);
          }
          umma_commit(&bars->s_full[buf]);
          if (done) umma_commit(&bars->q_empty[qb]);
          if (qt == nq - 1) umma_commit(&bars->k_empty[st]);
          ++cnt[t];
        }
      }
    }
  } else {
    const int t = (warp - 2) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t g = 0, cnt = 0;
    bool ok = true;
    for (int64_t it = begin; ok && it < end; ++it, ++g) {
      if ((g & 1) != static_cast<uint32_t>(t)) continue;
      const int h = static_cast<int>(it / tiles), kt = static_cast<int>(it - static_cast<int64_t>(h) * tiles);
      const int key = kt * TILE_KEYS + r;
      float acc = 0.f;
      for (int qt = 0; qt < nq; ++qt, ++cnt) {
        const uint32_t buf = 2 * t + (cnt & 1);
        const int rows = min(p.s.per_tile, p.s.n - qt * p.s.per_tile) * group;
        const float* nl = p.w.nlse + (static_cast<size_t>(h) * nq + qt) * TILE_ROWS;
        if (!warp_wait(&bars->s_full[buf], (cnt >> 1) & 1, v.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        float part[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < rows; c += 32) {
          uint32_t s[32];
          tmem_ld32(tmem + lane_off + buf * 128 + c, s);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            if (c + x >= rows) break;  // uniform
            const float n = nl[c + x];
            // rows that are not counted may hold anything
            part[x & 3] += n == -INFINITY ? 0.f : ex2(fmaf(__uint_as_float(s[x]), p.qscale, n));
          }
        }
        acc += (part[0] + part[1]) + (part[2] + part[3]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_free[buf]);
      }
      if (!ok) break;
      if (key < len) v.score[(static_cast<size_t>(p.a.prefix) * v.heads + h) * v.cap + key] += acc;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side
// The pool's stored vectors [slots, d]: boxes of one page's tokens x 64 channels.
cudaError_t page_map(CUtensorMap* m, const void* base, const PoolView& v) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(v.d),
                        static_cast<cuuint64_t>(v.pages) * v.heads * v.page};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(v.d) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(v.page)};
  cuuint32_t es[2] = {1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Queries [n][heads][group][d]: boxes of `entries` sequences' groups of one head x 64 channels.
cudaError_t query_map(CUtensorMap* m, const AttendArgs& a, int entries) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t d = a.v.d, g = a.group, h = a.v.heads;
  cuuint64_t dims[4] = {d, g, h, static_cast<cuuint64_t>(a.n)};
  cuuint64_t strides[3] = {d * 2, g * d * 2, h * g * d * 2};
  cuuint32_t box[4] = {64, static_cast<cuuint32_t>(a.group), 1, static_cast<cuuint32_t>(entries)};
  cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.q), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// A launch that may begin while the kernel before it drains.
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, int threads, size_t smem,
                         cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3(static_cast<unsigned>(threads));
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, args...);
}

template <int D>
cudaError_t attend_t(const Params& p, cudaStream_t stream) {
  CUtensorMap tq, t1, tk, tv;
  cudaError_t e;
  if ((e = query_map(&tq, p.a, p.s.per_tile)) != cudaSuccess) return e;
  if ((e = query_map(&t1, p.a, 1)) != cudaSuccess) return e;
  if ((e = page_map(&tk, p.a.v.K, p.a.v)) != cudaSuccess) return e;
  if ((e = page_map(&tv, p.a.v.V, p.a.v)) != cudaSuccess) return e;
  static int opted_in[kMaxDevices] = {}, opted_in_score[kMaxDevices] = {};
  if ((e = raise_smem_limit(reinterpret_cast<const void*>(pool_attend_kernel<D>), Cfg<D>::SMEM,
                            opted_in)) != cudaSuccess)
    return e;
  pool_attend_kernel<D><<<p.s.grid, kThreads, Cfg<D>::SMEM, stream>>>(tq, t1, tk, tv, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // enough blocks for the scores of few long rows: about four per SM
  const int rows = p.s.n * p.s.heads;
  const int chunks = p.a.accumulate
                         ? std::max(1, std::min(4 * p.s.grid / rows, (p.a.v.cap + 1023) / 1024))
                         : 1;
  if ((e = launch_after(pool_finish_kernel<D>, dim3(rows, chunks), kFinishThreads, 0, stream, p)) !=
      cudaSuccess)
    return e;
  if (!p.a.accumulate || p.a.prefix < 0) return cudaSuccess;
  if ((e = raise_smem_limit(reinterpret_cast<const void*>(pool_prefix_score_kernel<D>),
                            ScoreCfg<D>::SMEM, opted_in_score)) != cudaSuccess)
    return e;
  return launch_after(pool_prefix_score_kernel<D>, dim3(p.s.grid), kScoreThreads, ScoreCfg<D>::SMEM,
                      stream, tq, tk, p);
}

}  // namespace

size_t pool_attend_scratch(const AttendArgs& a) {
  if (a.v.kscale) return pool_attend_simple_scratch(a);
  return scratch_layout(shape_of(a, num_sms()), a.v.cap, a.accumulate, nullptr, nullptr);
}

cudaError_t pool_attend(const AttendArgs& a, void* scratch, cudaStream_t stream) {
  if (a.n == 0) return cudaSuccess;
  if (a.v.kscale) return pool_attend_simple(a, scratch, stream);
  Params p{};
  p.a = a;
  p.s = shape_of(a, num_sms());
  scratch_layout(p.s, a.v.cap, a.accumulate, scratch, &p.w);
  if (!a.accumulate) p.w.logits = nullptr;
  p.qscale = kLog2e / sqrtf(static_cast<float>(a.v.d));
  return a.v.d == 128 ? attend_t<128>(p, stream) : attend_t<64>(p, stream);
}

}  // namespace h2o
