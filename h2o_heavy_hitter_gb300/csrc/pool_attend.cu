// Attention of single tokens over the paged cache on the tensor cores: a prefix
// that the whole batch shares, then each sequence's own tokens. For row (b,
// query head) with key head h: s_j = q . k_j / sqrt(d), lse = log sum_j
// exp(s_j), p_j = exp(s_j - lse), out = sum_j p_j v_j; scores grow by p.
//
// Bound: every stored key and value is read from HBM once, 4 d bytes a token and
// head (2 d + 8 in E4M3), against 4 d flops per query row that sees it; below
// some 250 rows a head the bytes decide. So the kernels stream pages at full
// rate and keep the rest out of the way:
//
// pool_rows_kernel (here) takes units with at most 32 query rows: a sequence's
//   own tokens and one key head, with the head's query group as rows, and a
//   prefix whose rows (the groups of all sequences) are that few. The units'
//   128-key tiles form one list; a persistent CTA per SM takes an equal
//   contiguous share of it, whatever the lengths are: they are read on the device,
//   and every CTA finds its share with one scan. Rows are the narrow side of both
//   products, S^T = K Q^T (128 keys x rows) and O^T = V^T P^T (d x rows), so a
//   tile costs the tensor cores little more than feeding them, a thread owns one
//   key and has an exponential per row, and the accumulator is read out with a
//   thread per channel. (With rows as the wide side, 128 lanes of which 1 to 8
//   were used, the issue of both products and the read-out of the accumulator
//   took 2.9 us a tile against 1.5 us for its bytes.) Units alternate between two
//   warpgroups, so the end of one overlaps the beginning of the next. 256
//   sequences of 300 to 410 tokens, 32 heads of 128: 1.56 GB in 234 us (6.7 TB/s);
//   16 rows a head over 32768 tokens and the own ones: 0.70 GB in 120 us.
// pool_prefix_kernel, pool_prefix_score_kernel (pool_prefix.cu) take a prefix with
//   more rows.
// pool_finish_kernel joins the pieces of each row in fixed order and adds the
//   probabilities to the scores, from the logits that the first kernel left (4
//   bytes per key and row, against 4 d of keys and values).
//
// E4M3 pools: the codes of keys are matrix operands as they are, against queries
// split into two codes a value (pool_split_queries_kernel), with the key's and the
// row's scale applied to the logit; converting keys to bf16 too took 115 us where
// this took 110. Codes of values become bf16 in shared memory, by eight warps of
// their own, and their scales go into P. Bound by the work on a tile, not by its
// bytes: 64 sequences of up to 1000 tokens, 8 heads, 4 query heads each: 74 MB in 39 us.
//
// The second product takes P as two bf16 terms (split_bits): 16 significant bits,
// with an exponent that reaches as far as fp32's (a value's scale is in it). Logits,
// sums and accumulators are fp32. (One term, 8 bits, was the largest error of an
// output before its own rounding. The second costs the rows kernel next to nothing
// up to 16 rows and 15 % at 32, a prefix of 512 rows over 32768 keys 73 -> 92 us, the
// grouped E4M3 case above 76 -> 82 us in all.) What lies behind a sequence's
// end in its last page is not trusted: its probabilities are set to zero, and its
// values in shared memory too, since 0 times a NaN is not 0.
#include <algorithm>

#include "device_state.h"
#include "pool_tiles.cuh"

namespace h2o {
namespace {

// ------------------------------------------------------------------ the list of own tokens
struct List {
  int seq[kPoolMaxList];
  int len[kPoolMaxList];
  int cum[kPoolMaxList + 2];  // one more than used, for the alignment of what follows
};

// Fills the list: skipped and refused entries have seq -1 and no tiles. An entry
// is refused for an index outside the pool, the prefix's, or one named before;
// repeats are looked for one by one only where a hashed bit says that there may
// be some, or where the list is a later part of the caller's. Every CTA begins with
// this, so it takes few barriers. Blockwide; `bits`: 4 KB; `report`: this block sets
// the error word.
__device__ void build_list(const AttendArgs& a, List& list, uint32_t* bits, int* wsum,
                           bool report) {
  const PoolView& v = a.v;
  const int tid = threadIdx.x, nt = blockDim.x, n = a.n, lane = tid & 31, warp = tid >> 5;
  // each thread takes `per` entries in a row
  const int per = (n + nt - 1) / nt, b0 = min(n, tid * per), b1 = min(n, b0 + per);
  for (int b = b0; b < b1; ++b) {
    int s = a.seqs[b];
    if (s != -1 && (s < 0 || s >= v.seqs || s == a.prefix)) {
      if (report) atomicOr(v.err, kErrBadList);
      s = -1;
    }
    const int refused = s >= 0 ? __ldcg(v.refused + s) : 0;
    list.len[b] = s >= 0 ? checked_length(v, s, report) : -1;
    if (refused & kRefusedQueries) list.len[b] = -1;  // its row of the queries was not written
    list.seq[b] = s;
  }
  for (int i = tid; i < 1024; i += nt) bits[i] = 0;
  __syncthreads();
  bool seen = false;
  for (int b = b0; b < b1; ++b) {
    const int s = list.seq[b];
    if (s >= 0) seen |= (atomicOr(&bits[(s >> 5) & 1023], 1u << (s & 31)) >> (s & 31)) & 1u;
  }
  if (__syncthreads_or(seen || a.before)) {
    for (int b = b0; b < b1; ++b) {
      const int s = a.seqs[b];
      if (s < 0) continue;
      for (int j = -a.before; j < b; ++j)
        if (a.seqs[j] == s) {
          if (report) atomicOr(v.err, kErrBadList);
          list.len[b] = -1;
          break;
        }
    }
  }
  int mine = 0;
  for (int b = b0; b < b1; ++b) {
    if (list.len[b] < 0) list.seq[b] = -1;
    mine += key_tiles(max(0, list.len[b]));
  }
  int at = mine;  // inclusive over the warp, then over the block
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, at, off);
    if (lane >= off) at += y;
  }
  if (lane == 31) wsum[warp] = at;
  __syncthreads();
  for (int w = 0; w < warp; ++w) at += wsum[w];
  at -= mine;
  for (int b = b0; b < b1; ++b) {
    list.cum[b] = at;
    at += key_tiles(max(0, list.len[b]));
  }
  if (tid == nt - 1) list.cum[n] = at;
}

// A walk along one CTA's share of the units: first the prefix's (few rows only),
// one per head, then the own tokens'.
struct Walk {
  const AttendParams& p;
  const List& list;
  int plen, ptiles, cta;
  int64_t ptotal, at, end;
  // the unit: prefix or entry b, its key head, its sequence, its tiles in this share, its piece
  bool prefix;
  int h, b, seq, len, kt0, kt1, piece;

  __device__ Walk(const AttendParams& p, const List& list, int plen, int cta)
      : p(p), list(list), plen(plen), cta(cta) {
    ptiles = p.s.few ? key_tiles(plen) : 0;
    ptotal = static_cast<int64_t>(p.s.heads) * ptiles;
    const int64_t total = ptotal + static_cast<int64_t>(list.cum[p.s.n]) * p.s.heads;
    at = share_begin(total, p.s.grid, cta);
    end = share_begin(total, p.s.grid, cta + 1);
    b = -1;
  }
  __device__ int rows() const { return prefix ? p.s.n * p.s.group : p.s.group; }
  __device__ bool next() {
    if (at >= end) return false;
    int tiles;
    prefix = at < ptotal;
    if (prefix) {
      h = static_cast<int>(at / ptiles);
      kt0 = static_cast<int>(at - static_cast<int64_t>(h) * ptiles);
      seq = p.a.prefix;
      len = plen;
      tiles = ptiles;
      piece = h + cta;
    } else if (b < 0) {
      const int64_t q = at - ptotal;
      int lo = 0, hi = p.s.n - 1;  // the last entry that begins at or before q: the one with tiles
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
    } else {  // the next head, or the next entry with tiles
      kt0 = 0;
      if (++h == p.s.heads) {
        h = 0;
        do ++b;
        while (list.cum[b + 1] == list.cum[b]);
      }
      tiles = list.cum[b + 1] - list.cum[b];
    }
    if (!prefix) {
      seq = list.seq[b];
      len = list.len[b];
      piece = b * p.s.heads + h + cta;
    }
    kt1 = static_cast<int>(min(static_cast<int64_t>(tiles), kt0 + (end - at)));
    at += kt1 - kt0;
    return true;
  }
};

// The walk's tiles one by one.
struct TileCursor {
  Walk w;
  int kt, kt1, seq, len, h;
  __device__ explicit TileCursor(const Walk& walk) : w(walk), kt(-1), kt1(0) {}
  __device__ bool step() {
    if (++kt < kt1) return true;
    if (!w.next()) return false;
    kt = w.kt0;
    kt1 = w.kt1;
    seq = w.seq;
    len = w.len;
    h = w.h;
    return true;
  }
};

// ------------------------------------------------------------------ few rows
// Warps: 0 tiles of keys or codes by TMA, 1 MMA and TMEM, 2 queries, 3 tiles of
// values, 4..7 and 8..11 the two warpgroups, one per TMEM lane quadrant, 12..19
// E4M3 codes to bf16 tiles.
constexpr int kWarpMMA = 1, kWarpQ = 2, kWarpV = 3, kWarpRows = 4, kWarpCodes = 12;
constexpr int kCodeThreads = 256;
constexpr int kQBox = kFewRows * 128;  // rows x 64 channels (or keys) of an operand with few rows
constexpr int kSplitRows = 16;         // rows up to which one P operand holds both terms

template <int RK, int RV, int S>
struct Bars {
  RingBars<RK> keys;
  RingBars<RV> values;
  RingBars<S> codes;
  uint64_t q_full[2], q_empty[2];  // by unit
  uint64_t s_full[2][2];           // [warpgroup][buffer]
  uint64_t p_ready[2][2];
  uint64_t pv_done[2][2];
  uint64_t o_last[2], o_free[2];   // one phase per unit of the warpgroup
  uint64_t xbar[2];                // the warpgroup's exchange, a phase per use
  uint64_t drained;
  uint32_t tmem;
  int wsum[33];
  float xmax[2][2][4][kFewRows];   // [warpgroup][use & 1][quadrant][row]
};

template <int D, bool F8>
struct Cfg {
  static constexpr int THREADS = 32 * kWarpCodes + (F8 ? kCodeThreads : 0);
  static constexpr int TILE = TILE_KEYS * D * 2;
  static constexpr int KTILE = F8 ? TILE_KEYS * D : TILE;  // keys are used as they are stored
  static constexpr int RK = (F8 ? 3 : 2) * (128 / D), RV = (F8 ? 2 : 3) * (128 / D);
  static constexpr int S = F8 ? 2 * (128 / D) : 1;  // slots of value codes
  static constexpr int CODES = F8 ? S * TILE_KEYS * D : 0;
  static constexpr int Q = kQBox * (D / 64);  // a unit's queries; two buffers
  // A tile's probabilities, 128 keys x 32 columns: up to 16 rows' first terms and, kSplitRows
  // further, their second, two buffers per warpgroup; or, of more rows, the first terms in one
  // buffer and the second in the other.
  static constexpr int P = kQBox * 2;
  static constexpr int SCALES = F8 ? (RK + S + kScaleTiles) * TILE_KEYS * 4 : 0;
  static constexpr size_t SMEM = static_cast<size_t>(RK) * KTILE + RV * TILE + 2 * Q + 4 * P + CODES +
                                 SCALES + sizeof(List) + sizeof(Bars<RK, RV, S>) + 1024;
  // TMEM: S^T of warpgroup t in columns 64 t + 32 (0, 1), its O^T at 128 + 32 t
  static constexpr uint32_t O_COL = 128, TMEM_COLS = 256;
};

// Fp32 values as integers of the same order, for the integer maximum of a warp.
__device__ __forceinline__ int order_key(float x) {
  const int i = __float_as_int(x);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float order_value(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

// The sums over a warp of CH values per lane; lane i < CH gets value i's. Each
// step halves the values a lane holds, then what is left is summed over lanes.
template <int CH>
__device__ __forceinline__ float warp_sums(const float (&x)[CH], int lane) {
  float y[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) y[i] = x[i];
  int off = 16;
#pragma unroll
  for (int n = CH / 2; n >= 1; n /= 2, off /= 2) {
    const bool up = lane & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = up ? y[i] : y[i + n], keep = up ? y[i + n] : y[i];
      y[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
    }
  }
  float z = y[0];
#pragma unroll
  for (int o = 16 / CH; o; o /= 2) z += __shfl_xor_sync(0xffffffffu, z, o);
  // value i is in the lanes whose upper bits are i's, most significant first
  return CH == 1 ? z : __shfl_sync(0xffffffffu, z, (lane * (32 / CH)) & 31);
}

// One tile's logits and probabilities, thread = key.
struct TileRows {
  uint32_t s_tm;
  float ks, vs;   // scales of the key's logits and of its value
  float fac;      // E4M3: scale of row `lane`'s logits
  bool live;      // the key lies before the sequence's end
  uint8_t* p;     // row 0 of the P operand at this key's place in a 16-byte chunk
  int second;     // bytes from a row's first term to its second
  int chunk;      // that chunk
  float* logits;  // row 0's logit of this key, or null
  int cap, rows;
};

// Softmax of a tile against the running maximum m of row `lane`, CH rows at a
// time (unused ones are computed and dropped: branches would serialise the
// reductions). Raises m only where it grows by more than 2^8 (alpha, rescale);
// sum: row `lane`'s over this warp's keys. False: the exchange gave up.
template <int CH, bool F8, typename Exchange>
__device__ __forceinline__ bool tile_softmax(const TileRows& a, float& m, float& alpha,
                                             bool& rescale, float& sum, Exchange&& exchange) {
  const int lane = threadIdx.x & 31;
  uint32_t s[8];
  float mine = -INFINITY;
  for (int r0 = 0; r0 < a.rows; r0 += CH) {
    tmem_ld8(a.s_tm + r0, s);
    tmem_wait_ld();
    float top[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const float k = F8 ? a.ks * __shfl_sync(0xffffffffu, a.fac, r0 + i) : a.ks;
      const float z = a.live ? __uint_as_float(s[i]) * k : -INFINITY;
      top[i] = order_value(__reduce_max_sync(0xffffffffu, order_key(z)));
      if (a.logits && a.live && r0 + i < a.rows) a.logits[static_cast<size_t>(r0 + i) * a.cap] = z;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (lane == r0 + i) mine = top[i];
  }
  float all[4];
  if (!exchange(mine, all)) return false;
  const float mx = fmaxf(fmax3(all[0], all[1], all[2]), all[3]);
  alpha = 1.f;
  rescale = false;
  if (lane < a.rows && mx > m + 8.f) {
    rescale = m != -INFINITY;
    if (rescale) alpha = ex2(m - mx);
    m = mx;
  }
  const float ref = m == -INFINITY ? 0.f : m;
  sum = 0.f;
  for (int r0 = 0; r0 < a.rows; r0 += CH) {
    if (a.rows > CH) {
      tmem_ld8(a.s_tm + r0, s);
      tmem_wait_ld();
    }
    float pr[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const float n = __shfl_sync(0xffffffffu, ref, r0 + i);
      const float k = F8 ? a.ks * __shfl_sync(0xffffffffu, a.fac, r0 + i) : a.ks;
      pr[i] = a.live ? ex2(fmaf(__uint_as_float(s[i]), k, -n)) : 0.f;
      // K-major, 128-byte swizzle: 16-byte chunk (key / 8) of a row at chunk ^ (row & 7)
      const int row = r0 + i;
      uint8_t* at = a.p + row * 128 + ((a.chunk ^ (row & 7)) << 4);
      const uint32_t x = a.live ? split_bits<F8>(pr[i] * a.vs) : 0u;
      *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(x >> 16);
      *reinterpret_cast<__nv_bfloat16*>(at + a.second) = __float2bfloat16(__uint_as_float(x) - split_first(x));
    }
    const float x = __shfl_sync(0xffffffffu, warp_sums<CH>(pr, lane), (lane - r0) & 31);
    if (lane >= r0 && lane < r0 + CH) sum = x;
  }
  return true;
}

template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::THREADS, 1)
    pool_rows_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap t1,
                     const __grid_constant__ CUtensorMap tq2, const __grid_constant__ CUtensorMap t2,
                     const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                     const __grid_constant__ AttendParams p) {
  using C = Cfg<D, F8>;
  constexpr int RK = C::RK, RV = C::RV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sK = smem;
  uint8_t* sV = sK + RK * C::KTILE;
  uint8_t* sQ = sV + RV * C::TILE;
  uint8_t* sP = sQ + 2 * C::Q;
  uint8_t* codes = sP + 4 * C::P;
  float* kscales = reinterpret_cast<float*>(codes + C::CODES);  // [RK][128]
  float* cscales = kscales + RK * TILE_KEYS;                    // [S][128], of value codes
  float* vscales = cscales + C::S * TILE_KEYS;                  // [kScaleTiles][128]
  List& list = *reinterpret_cast<List*>(reinterpret_cast<uint8_t*>(kscales) + C::SCALES);
  auto* bars = reinterpret_cast<Bars<RK, RV, C::S>*>(&list + 1);
  const PoolView& v = p.a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  // beside the prefix kernel, which waited for what came before it and released that, this one
  // waits at its end
  if (p.a.prefix < 0 || p.s.few) {
    grid_dependency_wait();
  } else {
    if (threadIdx.x == 0) grid_acquire();
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < RK; ++i) {
      mbar_init(&bars->keys.full[i], 1);
      mbar_init(&bars->keys.empty[i], F8 ? 1 + 4 : 1);  // the product, and the readers of the scales
    }
    for (int i = 0; i < RV; ++i) {
      mbar_init(&bars->values.full[i], F8 ? kCodeThreads / 32 : 1);
      mbar_init(&bars->values.empty[i], 1);
    }
    for (int i = 0; i < C::S; ++i) {
      mbar_init(&bars->codes.full[i], 1);
      mbar_init(&bars->codes.empty[i], kCodeThreads / 32);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars->s_full[t][i], 1);
        mbar_init(&bars->p_ready[t][i], 4);
        mbar_init(&bars->pv_done[t][i], 1);
      }
      mbar_init(&bars->o_last[t], 1);
      mbar_init(&bars->o_free[t], 4);
      mbar_init(&bars->xbar[t], 4);
    }
    mbar_init(&bars->drained, 1);
    fence_barrier_init();
  }
  if (warp == kWarpMMA) {
    tmem_alloc(&bars->tmem, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == kWarpQ && lane == 0) {
    tma_prefetch_map(&tq);
    tma_prefetch_map(&t1);
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tk);
    tma_prefetch_map(&tv);
  }
  build_list(p.a, list, reinterpret_cast<uint32_t*>(sP), bars->wsum, cta == 0);
  const int plen = p.a.prefix >= 0 ? max(0, checked_length(v, p.a.prefix, cta + threadIdx.x == 0)) : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (cta == 0) {
    for (int i = threadIdx.x; i < p.s.n; i += C::THREADS) p.w.seq[i] = list.seq[i];
    for (int i = threadIdx.x; i <= p.s.n; i += C::THREADS) p.w.cum[i] = list.cum[i];
  }
  const uint32_t tmem = bars->tmem;
  Walk w(p, list, plen, cta);

  if (warp == 0) {
    if constexpr (F8)
      produce_codes<D, true>(v, &tk, v.kscale, sK, kscales, bars->keys, TileCursor(w));
    else
      produce_tma<D, true>(v, &tk, sK, bars->keys, TileCursor(w));
  } else if (warp == kWarpV) {
    if constexpr (F8)
      produce_codes<D, true>(v, &tv, v.vscale, codes, cscales, bars->codes, TileCursor(w));
    else
      produce_tma<D, true>(v, &tv, sV, bars->values, TileCursor(w));
  } else if (F8 && warp >= kWarpCodes) {
    convert_values<D, RV, C::S, kCodeThreads>(v, codes, cscales, bars->codes, sV, bars->values, vscales,
                                              TileCursor(w), threadIdx.x - 32 * kWarpCodes);
  } else if (warp == kWarpQ) {
    if (lane == 0) {
      uint32_t e = 0;
      for (; w.next(); ++e) {
        const int qb = e & 1;
        if (e >= 2 && !pool_wait(&bars->q_empty[qb], ((e >> 1) - 1) & 1, v.err)) break;
        mbar_arrive_expect_tx(&bars->q_full[qb], w.rows() * D * 2);
        // boxes of 64 channels, or the two codes of every value
#pragma unroll
        for (int c = 0; c < (F8 ? 2 : D / 64); ++c)
          tma_load_4d(sQ + qb * C::Q + c * (F8 ? kFewRows * D : kQBox),
                      c == 1 && F8 ? (w.prefix ? &tq2 : &t2) : (w.prefix ? &tq : &t1), F8 ? 0 : c * 64, 0,
                      w.h, w.prefix ? 0 : w.b, &bars->q_full[qb]);
      }
      drain_copies(bars->q_full, e, v.err);
    }
  } else if (warp == kWarpMMA) {
    // ---------------------------------------------------------------- MMA issuer
    // Tile g's S^T is followed by the O^T of tile g - 1, so that the softmax of
    // one overlaps the product of the next. An S^T buffer and a P buffer are those
    // of the warpgroup's tile before the last, whose O^T is issued by then; the
    // MMAs of one thread complete in order.
    {
      const uint64_t dk0 = F8 ? desc_codes<D>(sK) : desc_kmajor<D>(sK, 0);
      const uint64_t dq0 = F8 ? desc_codes<D>(sQ) : smem_desc(sQ, 16, 1024);
      const uint64_t dp0 = smem_desc(sP, 16, 1024);
      // V^T = the V tile with d as the long side of A (MN-major): 64 channels a box;
      // d = 64 has one box, which then serves as rows 64..127 too (not read)
      const uint64_t dv0 = smem_desc(sV, D == 128 ? kBoxBytes : 0, 1024);
      uint32_t g = 0, c[2] = {0, 0};  // tiles, and tiles of each warpgroup
      int e = 0;
      bool ok = true;
      struct {
        bool live = false, first, last, wide;
        int t, e;
        uint32_t c, g;
      } pv;
      constexpr uint32_t idesc_pv = idesc_bf16(TILE_KEYS, kFewRows, 0, 0) | (1u << 15);
      auto issue_pv = [&]() -> bool {
        const uint32_t st = pv.g % RV, buf = pv.c & 1;
        if (!pool_warp_wait(&bars->p_ready[pv.t][buf], (pv.c >> 1) & 1, v.err) ||
            !pool_warp_wait(&bars->values.full[st], (pv.g / RV) & 1, v.err) ||
            (pv.first && pv.e >= 2 && !pool_warp_wait(&bars->o_free[pv.t], ((pv.e >> 1) - 1) & 1, v.err)))
          return false;
        tc_fence_after();
        const uint64_t vb = dv0 + static_cast<uint64_t>(st * (C::TILE >> 4));
        const uint64_t pb = dp0 + static_cast<uint64_t>((pv.t * 2 + (pv.wide ? 0 : buf)) * (C::P >> 4));
        const uint32_t o = tmem + C::O_COL + pv.t * 32;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < TILE_KEYS / 16; ++kk)
            umma_ss(o, vb + kk * (2048 >> 4), pb + (((kk >> 2) * kQBox + (kk & 3) * 32) >> 4), idesc_pv,
                    (!pv.first || kk > 0) ? 1u : 0u);
          if (pv.wide) {
#pragma unroll
            for (int kk = 0; kk < TILE_KEYS / 16; ++kk)
              umma_ss(o, vb + kk * (2048 >> 4), pb + ((C::P + (kk >> 2) * kQBox + (kk & 3) * 32) >> 4),
                      idesc_pv, 1u);
          }
          umma_commit(&bars->values.empty[st]);
          umma_commit(&bars->pv_done[pv.t][buf]);
          if (pv.last) umma_commit(&bars->o_last[pv.t]);
        }
        __syncwarp();
        return true;
      };
      while (ok && w.next()) {
        const int t = e & 1, qb = e & 1;
        const int cols = w.rows() <= kSplitRows ? kSplitRows : kFewRows;
        const uint32_t idesc = idesc_bf16(TILE_KEYS, cols, 0, 0), idesc8 = idesc_e4m3(TILE_KEYS, cols);
        if (!pool_warp_wait(&bars->q_full[qb], (e >> 1) & 1, v.err)) break;
        for (int kt = w.kt0; kt < w.kt1; ++kt, ++g) {
          const uint32_t st = g % RK, buf = c[t] & 1;
          if (!pool_warp_wait(&bars->keys.full[st], (g / RK) & 1, v.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t kb = dk0 + static_cast<uint64_t>(st * (C::KTILE >> 4));
          const uint64_t qd = dq0 + static_cast<uint64_t>(qb * (C::Q >> 4));
          const uint32_t d_tm = tmem + t * 64 + buf * 32;
          if (elect_one()) {
            if constexpr (F8) {
#pragma unroll
              for (int kk = 0; kk < 2 * (D / 32); ++kk)  // the queries' first codes, then their second
                umma_ss_8bit(d_tm, kb + kk % (D / 32) * 2,
                             qd + kk / (D / 32) * (kFewRows * D >> 4) + kk % (D / 32) * 2, idesc8, kk > 0);
            } else {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                umma_ss(d_tm, kb + (((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4),
                        qd + (((kk >> 2) * kQBox + (kk & 3) * 32) >> 4), idesc, kk > 0);
            }
            umma_commit(&bars->s_full[t][buf]);
            umma_commit(&bars->keys.empty[st]);
            if (kt == w.kt1 - 1) umma_commit(&bars->q_empty[qb]);
          }
          __syncwarp();
          if (pv.live && !issue_pv()) {
            ok = false;
            break;
          }
          pv.live = true;
          pv.first = kt == w.kt0;
          pv.last = kt == w.kt1 - 1;
          pv.t = t;
          pv.e = e;
          pv.c = c[t]++;
          pv.g = g;
          pv.wide = w.rows() > kSplitRows;
        }
        ++e;
      }
      if (ok && pv.live) issue_pv();
      drain_products(&bars->drained, v.err);
    }
  } else if (warp >= kWarpRows && warp < kWarpCodes) {
    // ---------------------------------------------------------------- softmax
    // Thread = key r of the tile; lane i of every warp also keeps the running
    // maximum of row i (the same in the four warps) and the sum over its warp's keys.
    const int t = (warp - kWarpRows) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t o_tm = tmem + lane_off + C::O_COL + t * 32;
    uint32_t c = 0, g = 0, x = 0;  // tiles of this warpgroup, tiles, exchanges
    bool ok = true;
    // Every warp's 32 values to every warp of the group: returns the row of four of lane's.
    auto exchange = [&](float mine, float (&all)[4]) -> bool {
      float(*xm)[kFewRows] = bars->xmax[t][x & 1];
      xm[quad][lane] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->xbar[t]);
      if (!pool_warp_wait(&bars->xbar[t], x & 1, v.err)) return false;
      ++x;
#pragma unroll
      for (int i = 0; i < 4; ++i) all[i] = xm[i][lane];
      return true;
    };
    for (int e = 0; ok && w.next(); ++e) {
      if ((e & 1) != t) {
        g += w.kt1 - w.kt0;
        continue;
      }
      const int rows = w.rows();
      float* logits = nullptr;  // [rows][cap] of this unit
      if (w.prefix) {
        if (p.w.plogits) logits = p.w.plogits + static_cast<size_t>(w.h) * rows * v.cap;
      } else if (p.w.logits) {
        logits = p.w.logits + (static_cast<size_t>(w.b) * p.s.heads + w.h) * rows * v.cap;
      }
      const bool wide = rows > kSplitRows;
      float m = -INFINITY, l = 0.f;  // of row `lane`
      float fac = 1.f;               // E4M3: of row `lane`'s codes
      if (F8 && lane < rows)
        fac = p.w.qfac[w.prefix ? (static_cast<size_t>(lane / p.s.group) * p.s.heads + w.h) * p.s.group +
                                      lane % p.s.group
                                : (static_cast<size_t>(w.b) * p.s.heads + w.h) * p.s.group + lane];
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++g, ++c) {
        const uint32_t buf = c & 1, st = g % RV;
        const uint32_t s_tm = tmem + lane_off + t * 64 + buf * 32;
        const int valid = w.len - kt * TILE_KEYS;
        const bool live = r < valid;
        if (!pool_warp_wait(&bars->s_full[t][buf], (c >> 1) & 1, v.err)) {
          ok = false;
          break;
        }
        float ks = p.qscale, vs = 1.f;
        if (F8) {
          // the keys' product is done, so their tile has arrived; it stays until the arrival here
          if (!pool_warp_wait(&bars->keys.full[g % RK], (g / RK) & 1, v.err)) {
            ok = false;
            break;
          }
          ks *= kscales[g % RK * TILE_KEYS + r];
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->keys.empty[g % RK]);
        }
        if (F8 || valid < TILE_KEYS) {
          // the value tile stays in its slot until this warpgroup's probabilities are used
          if (!pool_warp_wait(&bars->values.full[st], (g / RV) & 1, v.err)) {
            ok = false;
            break;
          }
          if (F8) {
            vs = vscales[g % kScaleTiles * TILE_KEYS + r];
          } else {  // values behind the end count as zero, whatever they are
            for (int i = r; i < (TILE_KEYS - valid) * (D / 8); i += 128) {
              const int row = valid + i / (D / 8), ch = i % (D / 8);
              *reinterpret_cast<uint4*>(sV + st * C::TILE + (ch >> 3) * kBoxBytes + row * 128 +
                                        (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
          }
        }
        tc_fence_after();
        float alpha = 1.f, sum;
        bool rescale = false;
        const TileRows tr{s_tm, ks, vs, fac, live,
                          sP + (t * 2 + (wide ? 0 : buf)) * C::P + (r >> 6) * kQBox + (r & 7) * 2,
                          wide ? C::P : kSplitRows * 128, (r & 63) >> 3,
                          logits ? logits + kt * TILE_KEYS + r : nullptr, v.cap, rows};
        // many rows have one P buffer, which the O^T before this one must have read: it is
        // waited for behind the maximum
        auto maximum = [&](float mine, float (&all)[4]) -> bool {
          return exchange(mine, all) &&
                 (!wide || kt == w.kt0 ||
                  pool_warp_wait(&bars->pv_done[t][(c - 1) & 1], ((c - 1) >> 1) & 1, v.err));
        };
        const bool done = rows == 1   ? tile_softmax<1, F8>(tr, m, alpha, rescale, sum, exchange)
                          : rows <= 4 ? tile_softmax<4, F8>(tr, m, alpha, rescale, sum, exchange)
                                      : tile_softmax<8, F8>(tr, m, alpha, rescale, sum, maximum);
        if (!done) {
          ok = false;
          break;
        }
        l = fmaf(l, alpha, sum);
        if (__any_sync(0xffffffffu, rescale)) {  // the same in the four warps
          // the O^T before this one must be complete
          if (!pool_warp_wait(&bars->pv_done[t][(c - 1) & 1], ((c - 1) >> 1) & 1, v.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int r0 = 0; r0 < rows; r0 += 8) {
            for (int term = 0; term < (wide ? 1 : 2); ++term) {
              uint32_t o[8];
              tmem_ld8(o_tm + term * kSplitRows + r0, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(0xffffffffu, alpha, (r0 + i) & 31));
              tmem_st8(o_tm + term * kSplitRows + r0, o);
            }
          }
          tmem_wait_st();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_ready[t][buf]);
      }
      if (!ok) break;
      // ---- the piece
      float part[4];
      if (!exchange(l, part)) break;
      l = (part[0] + part[1]) + (part[2] + part[3]);
      if (!pool_warp_wait(&bars->o_last[t], (e >> 1) & 1, v.err)) break;
      tc_fence_after();
      const size_t rec = static_cast<size_t>(w.piece) * (w.prefix ? kFewRows : p.s.group);
      float* out = (w.prefix ? p.w.po : p.w.to) + rec * D;
      for (int r0 = 0; r0 < rows; r0 += 8) {
        uint32_t o[8], o2[8];
        tmem_ld8(o_tm + r0, o);
        if (!wide) tmem_ld8(o_tm + kSplitRows + r0, o2);
        tmem_wait_ld();
        if (r < D) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (r0 + i >= rows) break;
            out[(r0 + i) * D + r] = __uint_as_float(o[i]) + (wide ? 0.f : __uint_as_float(o2[i]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_free[t]);
      if (quad == 0 && lane < rows)
        (w.prefix ? p.w.pml : p.w.tml)[rec + lane] = make_float2(m, l);
    }
  }
  // the prefix kernel may still run: what follows waits for both (pool_prefix_score_kernel
  // begins with keys and queries, which are older than both)
  if (p.a.prefix < 0 || p.s.few)
    grid_launch_dependents();
  else if (threadIdx.x == 0)
    grid_release_dependents();
  grid_dependency_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------------ queries of an E4M3 pool
// A query row as two E4M3 codes a value, x = fac (first + second): the row is
// scaled by a power of two to a magnitude in [128, 256); the first code has the
// upper four of a bf16 value's eight significant bits, the second what is left,
// down to steps of 2^-9: no more than 2^-17 of the row's largest value is lost in
// any value (2^-136 where the largest is below 2^-119: the power of two ends at 2^126,
// whose reciprocal fp32 still holds in full). A row with an infinity or a NaN gets a
// NaN for its factor. A warp per row.
template <int D>
__global__ void __launch_bounds__(256)
    pool_split_queries_kernel(const __nv_bfloat16* __restrict__ q, int rows, uint8_t* q8, float* qfac) {
  constexpr int N = D / 32;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  if (row >= rows) return;
  uint32_t raw[N / 2];
  if constexpr (N == 4)
    *reinterpret_cast<uint2*>(raw) = reinterpret_cast<const uint2*>(q + static_cast<size_t>(row) * D)[lane];
  else
    raw[0] = reinterpret_cast<const uint32_t*>(q + static_cast<size_t>(row) * D)[lane];
  float x[N], amax = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = __uint_as_float(i & 1 ? raw[i / 2] & 0xffff0000u : raw[i / 2] << 16);
    amax = fmaxf(amax, fabsf(x[i]));
  }
  bool wild = false;
#pragma unroll
  for (int i = 0; i < N; ++i) wild |= !(fabsf(x[i]) < INFINITY);
#pragma unroll
  for (int off = 16; off; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  wild = __any_sync(0xffffffffu, wild);
  // 2^(7 - exponent of amax), within fp32's normal numbers
  const int e = min(max(7 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127), -126), 126);
  const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
  uint32_t codes[2] = {0, 0};  // this lane's N codes of each half
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float a = x[i] * up, b = x[i + 1] * up;
    const uint32_t hi = f32x2_to_e4m3x2(a, b);
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
    codes[0] |= hi << (8 * i);
    codes[1] |= f32x2_to_e4m3x2(a - f.x, b - f.y) << (8 * i);
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint8_t* out = q8 + (static_cast<size_t>(half) * rows + row) * D + lane * N;
    if constexpr (N == 4)
      *reinterpret_cast<uint32_t*>(out) = codes[half];
    else
      *reinterpret_cast<uint16_t*>(out) = static_cast<uint16_t>(codes[half]);
  }
  if (lane == 0)
    qfac[row] = wild ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// ------------------------------------------------------------------ joining the pieces
constexpr int kFinishWarps = 4, kFinishThreads = 32 * kFinishWarps;

// place_records by L adjacent lanes: the four divisions run in as many of them.
template <int L>
__device__ __forceinline__ Records records_of(const AttendParams& p, int b, int h, int plen,
                                              const int (&cum)[3], int lane) {
  return place_records(p, b, h, plen, cum, [&](const int64_t (&at)[4], const int64_t (&total)[2], int (&c)[4]) {
    const int64_t x = lane == 0 ? at[0] : lane == 1 ? at[1] : lane == 2 ? at[2] : at[3];
    const int64_t n = lane < 2 ? total[0] : total[1];
    const int mine = n > 0 ? owner(x, n, p.s.grid) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __shfl_sync(0xffffffffu, mine, i, L);
  });
}

// The lse (base 2) of row g by L adjacent lanes (all groups of a warp at once), the
// same bits in every block; `first`: the maximum of record `lane`.
template <int L, bool L2>
__device__ __forceinline__ float row_lse(const AttendParams& p, const Records& x, int g, int lane,
                                         float& first) {
  const int all = x.prefix + x.own;
  float m = -INFINITY, l = 0.f;
  first = -INFINITY;
#pragma unroll 2
  for (int i = lane; i < all; i += L) {
    const float2 y = record_ml<L2>(p, x, i, g);
    if (i < L) first = y.x;
    join(m, l, y.x, y.y);
  }
#pragma unroll
  for (int off = L / 2; off; off >>= 1) {
    const float mo = __shfl_xor_sync(0xffffffffu, m, off), lo = __shfl_xor_sync(0xffffffffu, l, off);
    join(m, l, mo, lo);
  }
  return __shfl_sync(0xffffffffu, all ? m + log2f(l) : -INFINITY, 0, L);
}

// Scores of a prefix with few rows, from their logits, rows in order: a block per
// head and 4 kFinishThreads keys. It computes the lse's of all rows itself, which
// takes less than another launch would.
__device__ void prefix_scores(const AttendParams& p, int block, float* s_lse) {
  const PoolView& v = p.a.v;
  const int per_head = (v.cap + 4 * kFinishThreads - 1) / (4 * kFinishThreads);
  const int h = block / per_head, j = ((block - h * per_head) * kFinishThreads + threadIdx.x) * 4;
  const int plen = max(0, checked_length(v, p.a.prefix, false));
  if ((block - h * per_head) * kFinishThreads * 4 >= plen) return;
  // eight lanes a row (a warp a row, of 16 rows, took 6 us longer over 32 heads of 32768 keys)
  const int rows = p.s.n * p.s.group, lane = threadIdx.x & 7;
  for (int i0 = 0; i0 < rows; i0 += kFinishThreads / 8) {
    const int i = i0 + (threadIdx.x >> 3), b = min(i, rows - 1) / p.s.group;
    const int cum[3] = {p.w.cum[b], p.w.cum[b + 1], p.w.cum[p.s.n]};
    float first;
    const float x = row_lse<8, false>(p, records_of<8>(p, b, h, plen, cum, lane),
                                      min(i, rows - 1) - b * p.s.group, lane, first);
    // +inf: not counted, whatever its logits are
    if (lane == 0 && i < rows) s_lse[i] = p.w.seq[b] < 0 ? INFINITY : x;
  }
  __syncthreads();
  if (j >= plen) return;
  const float* L = p.w.plogits + static_cast<size_t>(h) * rows * v.cap + j;
  float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = 0; i < rows; ++i) {
    const float n = s_lse[i];
    const float4 y = *reinterpret_cast<const float4*>(L + static_cast<size_t>(i) * v.cap);
    if (n == INFINITY) continue;
    a[0] += ex2(y.x - n);
    a[1] += ex2(y.y - n);
    a[2] += ex2(y.z - n);
    a[3] += ex2(y.w - n);
  }
  float* score = v.score + (static_cast<size_t>(p.a.prefix) * v.heads + h) * v.cap + j;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (j + i < plen) score[i] += a[i];
}

// Per (entry, key head) and chunk of keys, one to four warps by the size of the
// group (unit_warps; a row each at a time): join the rows, a warp each, in the order of
// the pieces, and add the probabilities of the own tokens to their scores. Every
// chunk computes the lse's it needs, chunk 0 writes. `blocks` * `chunks` such blocks,
// then those of the prefix's scores. Latency-bound: the lengths, the records, then
// the outputs are loads behind one another; 8192 rows take 20 us, 4 rows 6.
template <int D, bool L2>
__device__ __forceinline__ void finish_block(const AttendParams& p, int unit_warps, int blocks, int chunks,
                                             float (&s_lse)[kFinishWarps][kFewRows]) {
  const PoolView& v = p.a.v;
  const int group = p.s.group, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x / blocks, block = blockIdx.x - chunk * blocks;
  const int local = warp / unit_warps, sub = warp - local * unit_warps;
  const int unit = block * (kFinishWarps / unit_warps) + local;
  const bool in = unit < p.s.n * p.s.heads;
  const int b = in ? unit / p.s.heads : 0, h = in ? unit - b * p.s.heads : 0;
  const int cum[3] = {load<L2>(p.w.cum + b), load<L2>(p.w.cum + b + 1), load<L2>(p.w.cum + p.s.n)};
  const int seq = in ? load<L2>(p.w.seq + b) : -1;
  const int plen = p.a.prefix >= 0 ? max(0, checked_length(v, p.a.prefix, false)) : 0;
  float* nlse = nullptr;  // for the scores of a prefix with many rows
  if (in && p.w.nlse && chunk == 0)
    nlse = p.w.nlse + (static_cast<size_t>(h) * p.s.nq + b / p.s.per_tile) * TILE_ROWS +
           b % p.s.per_tile * group;
  int len = 0;
  if (seq >= 0) {
    len = load<L2>(v.meta + 2 * seq);
    const Records x = records_of<32>(p, b, h, plen, cum, lane);
    const int all = x.prefix + x.own;
    for (int g = sub; g < group; g += unit_warps) {
      float first;
      const float lse = row_lse<32, L2>(p, x, g, lane, first);
      if (lane == 0) s_lse[local][g] = lse;
      if (chunk) continue;
      float acc[D / 32] = {};
      for (int i0 = 0; i0 < all; i0 += 32) {
        const float mine =
            i0 == 0 ? first : i0 + lane < all ? record_ml<L2>(p, x, i0 + lane, g).x : -INFINITY;
        const float wgt = all ? ex2(mine - lse) : 0.f;
        const int n = min(32, all - i0);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
          const float wi = __shfl_sync(0xffffffffu, wgt, i);
          const float* o = (i0 + i < x.prefix ? p.w.po : p.w.to) +
                           record(p, x, i0 + i, g) * D + lane * (D / 32);
          float part[D / 32];
          if constexpr (D == 128) {
            const float4 y = load<L2>(reinterpret_cast<const float4*>(o));
            part[0] = y.x, part[1] = y.y, part[2] = y.z, part[3] = y.w;
          } else {
            const float2 y = load<L2>(reinterpret_cast<const float2*>(o));
            part[0] = y.x, part[1] = y.y;
          }
#pragma unroll
          for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(wi, part[c], acc[c]);
        }
      }
      const size_t row = static_cast<size_t>(unit) * group + g;
      uint32_t* out = static_cast<uint32_t*>(p.a.out) + row * (D / 2) + lane * (D / 64);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) out[c] = pack_bf16x2(acc[2 * c], acc[2 * c + 1]);
      if (lane == 0) {
        if (p.a.lse) p.a.lse[row] = lse * 0.69314718055994531f;  // ln 2
        if (nlse) nlse[g] = -lse;
      }
    }
  } else if (nlse && sub == 0 && lane < group) {
    nlse[lane] = -INFINITY;
  }
  if (!p.w.logits) return;
  __syncthreads();
  if (seq < 0) return;
  const float* L = p.w.logits + static_cast<size_t>(unit) * group * v.cap;
  float* score = v.score + (static_cast<size_t>(seq) * v.heads + h) * v.cap;
  const int step = chunks * unit_warps * 128;
  for (int j = ((chunk * unit_warps + sub) * 32 + lane) * 4; j < len; j += step) {
    // four slots a lane: a sequence's rows end at a multiple of its page
    float4 sum = load<L2>(reinterpret_cast<const float4*>(score + j));
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int g = 0; g < group; ++g) {
      const float4 y = load<L2>(reinterpret_cast<const float4*>(L + static_cast<size_t>(g) * v.cap + j));
      const float n = s_lse[local][g];
      a[0] += ex2(y.x - n);
      a[1] += ex2(y.y - n);
      a[2] += ex2(y.z - n);
      a[3] += ex2(y.w - n);
    }
    sum.x += a[0];
    if (j + 1 < len) sum.y += a[1];
    if (j + 2 < len) sum.z += a[2];
    if (j + 3 < len) sum.w += a[3];
    *reinterpret_cast<float4*>(score + j) = sum;
  }
}

// `beside`: launched behind pool_prefix_score_kernel, whose trigger stands behind its wait for
// the kernels that left the pieces. This one reads nothing of that kernel, so only its own end
// waits: what follows this kernel follows both. Without a wait nothing is promised of this SM's
// L1, so what others wrote is read from L2 (load<true>), where those kernels, complete, have left it.
// (An acquire by each of the 2048 blocks of 256 sequences x 32 heads cost 3 us.)
template <int D, bool beside>
__global__ void __launch_bounds__(kFinishThreads)
    pool_finish_kernel(const __grid_constant__ AttendParams p, int unit_warps, int blocks, int chunks) {
  __shared__ float s_lse[kFinishWarps][kFewRows];
  if (!beside) grid_dependency_wait();
  if (!p.w.nlse)
    grid_launch_dependents();
  else if (threadIdx.x == 0)  // the score kernel follows, and begins with keys and queries
    grid_release_dependents();
  if (static_cast<int>(blockIdx.x) >= blocks * chunks)
    prefix_scores(p, blockIdx.x - blocks * chunks, s_lse[0]);
  else
    finish_block<D, beside>(p, unit_warps, blocks, chunks, s_lse);
  if (beside && blockIdx.x == 0) grid_dependency_wait();
}

// ------------------------------------------------------------------ host side
Shape shape_of(const AttendArgs& a, int sms) {
  Shape s{};
  s.n = a.n;
  s.heads = a.v.heads;
  s.group = a.group;
  s.d = a.v.d;
  s.few = a.prefix >= 0 && a.n * a.group <= kFewRows;
  s.per_tile = s.few ? a.n : TILE_ROWS / a.group;
  s.nq = (a.n + s.per_tile - 1) / s.per_tile;
  s.blocks = a.prefix >= 0 ? (s.nq + 1) / 2 : 0;
  s.grid = sms;
  return s;
}

size_t scratch_layout(const Shape& s, int cap, bool accumulate, bool codes, void* base,
                      AttendScratch* out) {
  size_t at = 0;
  auto take = [&](size_t bytes) -> char* {
    if (!bytes) return nullptr;
    char* x = static_cast<char*>(base) + at;
    at += (bytes + 255) / 256 * 256;
    return x;
  };
  const size_t pieces = static_cast<size_t>(s.heads) * s.blocks + s.grid;
  const size_t prow = s.blocks ? pieces * (s.few ? kFewRows : 2 * TILE_ROWS) : 0;
  const size_t trow = (static_cast<size_t>(s.n) * s.heads + s.grid) * s.group;
  const size_t all = static_cast<size_t>(s.n) * s.heads * s.group;
  AttendScratch w{};
  w.seq = reinterpret_cast<int*>(take(s.n * sizeof(int)));
  w.cum = reinterpret_cast<int*>(take((s.n + 1) * sizeof(int)));
  const bool nlse = s.blocks && !s.few && accumulate && !score_joins(s);
  w.nlse = reinterpret_cast<float*>(
      take(nlse ? static_cast<size_t>(s.heads) * s.nq * TILE_ROWS * sizeof(float) : 0));
  w.pml = reinterpret_cast<float2*>(take(prow * sizeof(float2)));
  w.tml = reinterpret_cast<float2*>(take(trow * sizeof(float2)));
  w.po = reinterpret_cast<float*>(take(prow * s.d * sizeof(float)));
  w.to = reinterpret_cast<float*>(take(trow * s.d * sizeof(float)));
  w.logits = reinterpret_cast<float*>(take(accumulate ? all * cap * sizeof(float) : 0));
  w.plogits = reinterpret_cast<float*>(take(accumulate && s.few ? all * cap * sizeof(float) : 0));
  w.q8 = reinterpret_cast<uint8_t*>(take(codes ? 2 * all * s.d : 0));
  w.qfac = reinterpret_cast<float*>(take(codes ? all * sizeof(float) : 0));
  if (out) *out = w;
  return at;
}

template <int D, bool F8>
cudaError_t attend_t(const AttendParams& p, cudaStream_t stream) {
  CUtensorMap tq, t1, tq2, t2;  // tq: for a prefix with few rows only; the second codes: E4M3 only
  const CUtensorMap &tk = *p.a.kmap, &tv = *p.a.vmap;
  cudaError_t e;
  if (F8) {
    if ((e = pool_split_queries(p, stream)) != cudaSuccess) return e;
    if ((e = query_code_map(&t1, p, 0, 1)) != cudaSuccess) return e;
    if ((e = query_code_map(&t2, p, 1, 1)) != cudaSuccess) return e;
  } else {
    if ((e = query_map(&t1, p.a, 1)) != cudaSuccess) return e;
    t2 = t1;
  }
  tq = t1;
  tq2 = t2;
  if (p.s.few) {
    e = F8 ? query_code_map(&tq, p, 0, p.s.n) : query_map(&tq, p.a, p.s.n);
    if (e == cudaSuccess && F8) e = query_code_map(&tq2, p, 1, p.s.n);
    if (e != cudaSuccess) return e;
  }
  const bool many = p.a.prefix >= 0 && !p.s.few;
  if (many && (e = pool_prefix(p, stream)) != cudaSuccess) return e;
  using C = Cfg<D, F8>;
  static int opted_in[kMaxDevices] = {};
  if ((e = raise_smem_limit(reinterpret_cast<const void*>(pool_rows_kernel<D, F8>), C::SMEM,
                            opted_in)) != cudaSuccess)
    return e;
  if ((e = launch_after(pool_rows_kernel<D, F8>, dim3(p.s.grid), C::THREADS, C::SMEM, stream, tq, t1, tq2,
                        t2, tk, tv, p)) != cudaSuccess)
    return e;
  const int unit_warps = p.s.group >= 4 ? 4 : p.s.group >= 2 ? 2 : 1, units = p.s.n * p.s.heads;
  const int blocks = (units * unit_warps + kFinishWarps - 1) / kFinishWarps;
  // enough chunks of keys for the scores of few long rows
  const int chunks = p.a.accumulate
                         ? std::max(1, std::min(8 * p.s.grid / blocks, (p.a.v.cap + 511) / 512))
                         : 1;
  const int per_block = 4 * kFinishThreads;  // keys of prefix_scores
  const int sums = p.w.plogits ? p.s.heads * ((p.a.v.cap + per_block - 1) / per_block) : 0;
  const bool scores = many && p.a.accumulate, beside = scores && score_joins(p.s);
  if (beside && (e = pool_prefix_score(p, stream)) != cudaSuccess) return e;
  if ((e = launch_after(beside ? pool_finish_kernel<D, true> : pool_finish_kernel<D, false>,
                        dim3(blocks * chunks + sums), kFinishThreads, 0, stream, p, unit_warps, blocks,
                        chunks)) != cudaSuccess)
    return e;
  return scores && !beside ? pool_prefix_score(p, stream) : cudaSuccess;
}

}  // namespace

namespace {
cudaError_t encode(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base,
                   const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
                   CUtensorMapSwizzle swizzle) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint32_t es[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, type, rank, const_cast<void*>(base), dims, strides, box, es,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Swizzle of E4M3 operands with rows of d bytes.
CUtensorMapSwizzle code_swizzle(int d) {
  return d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
}

cudaError_t queries(CUtensorMap* m, const AttendArgs& a, int entries, const void* base, bool codes) {
  const cuuint64_t d = a.v.d, g = a.group, h = a.v.heads, row = codes ? d : 2 * d;
  const cuuint64_t dims[4] = {d, g, h, static_cast<cuuint64_t>(a.n)};
  const cuuint64_t strides[3] = {row, g * row, h * g * row};
  const cuuint32_t box[4] = {codes ? static_cast<cuuint32_t>(d) : 64, static_cast<cuuint32_t>(a.group), 1,
                             static_cast<cuuint32_t>(entries)};
  return encode(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims,
                strides, box, codes ? code_swizzle(a.v.d) : CU_TENSOR_MAP_SWIZZLE_128B);
}
}  // namespace

cudaError_t pool_page_map(CUtensorMap* m, const PoolView& v, bool keys) {
  const bool codes = v.kscale != nullptr;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(v.d),
                              static_cast<cuuint64_t>(v.pages) * v.heads * v.page};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(v.row_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(codes ? v.d : 64), static_cast<cuuint32_t>(v.page)};
  return encode(m, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                keys ? v.K : v.V, dims, strides, box,
                !codes ? CU_TENSOR_MAP_SWIZZLE_128B : keys ? code_swizzle(v.d) : CU_TENSOR_MAP_SWIZZLE_NONE);
}

cudaError_t query_map(CUtensorMap* m, const AttendArgs& a, int entries) {
  return queries(m, a, entries, a.q, false);
}

cudaError_t query_code_map(CUtensorMap* m, const AttendParams& p, int half, int entries) {
  const size_t rows = static_cast<size_t>(p.s.n) * p.s.heads * p.s.group;
  return queries(m, p.a, entries, p.w.q8 + half * rows * p.s.d, true);
}

cudaError_t pool_split_queries(const AttendParams& p, cudaStream_t stream) {
  const int rows = p.s.n * p.s.heads * p.s.group;
  return launch_after(p.s.d == 128 ? pool_split_queries_kernel<128> : pool_split_queries_kernel<64>,
                      dim3((rows + 7) / 8), 256, 0, stream, static_cast<const __nv_bfloat16*>(p.a.q), rows,
                      p.w.q8, p.w.qfac);
}

size_t pool_attend_scratch(const AttendArgs& a) {
  return scratch_layout(shape_of(a, num_sms()), a.v.cap, a.accumulate, a.v.kscale, nullptr, nullptr);
}

cudaError_t pool_attend(const AttendArgs& a, void* scratch, cudaStream_t stream) {
  if (a.n == 0) return cudaSuccess;
  AttendParams p{};
  p.a = a;
  p.s = shape_of(a, num_sms());
  scratch_layout(p.s, a.v.cap, a.accumulate, a.v.kscale, scratch, &p.w);
  p.qscale = kLog2e / sqrtf(static_cast<float>(a.v.d));
  if (a.v.kscale) return a.v.d == 128 ? attend_t<128, true>(p, stream) : attend_t<64, true>(p, stream);
  return a.v.d == 128 ? attend_t<128, false>(p, stream) : attend_t<64, false>(p, stream);
}

}  // namespace h2o
