// Shared parts of the paged attention kernels: the scratch of a call, the list
// of 128-key tiles that CTAs share, and the producers that bring tiles of keys
// and values into shared memory as bf16 matrix operands.
#pragma once

#include "common.cuh"
#include "device_state.h"
#include "kernels.h"
#include "pool.h"
#include "scan.cuh"
#include "tc.cuh"

namespace h2o {

constexpr int TILE_KEYS = 128;
constexpr int TILE_ROWS = 128;
constexpr int kFewRows = 32;  // query rows of a head that the few-rows kernel takes

// ------------------------------------------------------------------ a call
// Host-computed shape.
struct Shape {
  int n, heads, group, d;
  // The prefix has at most kFewRows query rows per head. Narrow against wide rows, us a
  // call (E4M3): 16 rows x 32 heads over 32768 keys 129 against 169 (151 against 187), 24
  // rows 164 against 173 (198, 192), 32 rows 211 against 173 (250, 196) there; but 43 against
  // 50 (52, 55) as 8 heads of groups of 4 and 43 against 54 (50, 62) as 8 heads of groups of
  // 8 over 8192 keys and 1000 own tokens each. The lengths, which would decide, are on the device.
  bool few;
  int per_tile;  // sequences whose query groups share a tile of rows of the prefix
  int nq;        // row tiles per head
  int blocks;    // prefix units per head: blocks of two row tiles (0 without a prefix)
  int grid;      // CTAs of the attention kernels
};

// Scratch, in order of allocation. A "piece" is what one CTA computed of one
// unit of tiles: per row an unnormalised output, a maximum and a sum. Piece u + c
// belongs to unit u and CTA c, unique since both only grow along the list.
struct AttendScratch {
  int* seq;        // [n] sequence of an entry, -1 skipped
  int* cum;        // [n + 1] own tiles of the entries before
  float* nlse;     // [heads][nq][128] -lse (base 2) of a prefix row, -inf: not counted
                   // (accumulate, unless score_joins)
  float2* pml;     // prefix pieces {max, sum}: many rows [heads * blocks + grid][2][128],
                   // few rows [heads + grid][kFewRows]
  float2* tml;     // own pieces [n * heads + grid][group]
  float* po;       // prefix pieces' outputs, [d] per row
  float* to;       // own pieces' outputs
  float* logits;   // [n][heads][group][cap] base-2 logits of the own tokens (accumulate only)
  float* plogits;  // [heads][n * group][cap] of the prefix (accumulate, few rows only)
  uint8_t* q8;     // E4M3 pool: the queries as two codes each, [2][n][heads][group][d]
  float* qfac;     // and what a row's codes are to be multiplied by, [n][heads][group]
};

struct AttendParams {
  AttendArgs a;
  Shape s;
  AttendScratch w;
  float qscale;  // log2(e) / sqrt(d)
};

// The prefix's score kernel joins the sums of its rows itself, and runs beside the
// finish kernel, where two row tiles hold them. Beyond, every CTA would do that for
// all rows of a head and keep them; it follows the finish kernel, which leaves them
// in AttendScratch::nlse.
inline __host__ __device__ bool score_joins(const Shape& s) { return s.nq <= 2; }

// Launchers of the kernels for a prefix with many rows (pool_prefix.cu). The
// first leaves pieces, the second adds the prefix's scores.
cudaError_t pool_prefix(const AttendParams& p, cudaStream_t stream);
cudaError_t pool_prefix_score(const AttendParams& p, cudaStream_t stream);
// Tensor map of the queries [n][heads][group][d] in boxes of `entries` groups of
// one head x 64 channels, or of one half of their codes (0, 1) x all channels
// (pool_attend.cu).
cudaError_t query_map(CUtensorMap* m, const AttendArgs& a, int entries);
cudaError_t query_code_map(CUtensorMap* m, const AttendParams& p, int half, int entries);

#ifdef __CUDACC__
// ------------------------------------------------------------------ bounded waits
// mbar_wait with its loop out of line: these kernels run some dozen waits in as
// many roles at once, and their code shares the instruction cache.
static __device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, int32_t* err) {
  return mbar_wait(bar, parity, err);
}
__device__ __forceinline__ bool pool_wait(uint64_t* bar, uint32_t parity, int32_t* err) {
  return mbar_try_wait(bar, parity) || wait_on(bar, parity, err);
}
// A role that filled slots of a ring of R `count` times in all, in order, waits for its copies
// in flight before it leaves, whoever gave up: the CTA's shared memory may be another's then.
// When nobody did, they are what the consumers wait for. One thread, or a whole warp. (Both out
// of line: in line they cost the E4M3 kernels 3 us.)
static __device__ __noinline__ void drain_ring(uint64_t* full, uint32_t ring, uint32_t count, int32_t* err) {
  for (uint32_t i = count > ring ? count - ring : 0; i < count; ++i)
    mbar_wait(&full[i % ring], (i / ring) & 1, err);
}
template <int R>
__device__ __forceinline__ void drain_copies(uint64_t (&full)[R], uint32_t count, int32_t* err) {
  drain_ring(full, R, count, err);
}
// The warp that issued products waits until none is left, before the CTA frees their TMEM.
// `bar`: one phase of one arrival.
static __device__ __noinline__ void drain_products(uint64_t* bar, int32_t* err) {
  __syncwarp();
  if (elect_one()) umma_commit(bar);
  __syncwarp();
  mbar_wait(bar, 0, err);
  __syncwarp();
}
// The result is made warp-uniform (see warp_wait).
__device__ __forceinline__ bool pool_warp_wait(uint64_t* bar, uint32_t parity, int32_t* err) {
  return __all_sync(0xffffffffu, pool_wait(bar, parity, err));
}

// ------------------------------------------------------------------ lengths, shares
// A load, L2: past L1.
template <bool L2, typename T>
__device__ __forceinline__ T load(const T* at) {
  return L2 ? __ldcg(at) : *at;
}

// A sequence's length, -1 (reported when `report`) for a state that no call leaves.
__device__ __forceinline__ int checked_length(const PoolView& v, int seq, bool report) {
  const int len = __ldcg(v.meta + 2 * seq);
  if (len >= 0 && len <= v.cap) return len;
  if (report) atomicOr(v.err, kErrBadState);
  return -1;
}

__device__ __forceinline__ int key_tiles(int len) { return (len + TILE_KEYS - 1) / TILE_KEYS; }

// CTAs that get a share of `total` tiles: none is left without one between two that have.
__device__ __forceinline__ int64_t sharers(int64_t total, int grid) {
  return min(total, static_cast<int64_t>(grid));
}

// First tile of CTA `cta`'s share of `total` tiles; the share ends where the next one's begins.
__device__ __forceinline__ int64_t share_begin(int64_t total, int grid, int cta) {
  const int64_t c = sharers(total, grid);
  return cta < c ? total * cta / c : total;
}

// CTA whose share holds tile `at`.
__device__ __forceinline__ int owner(int64_t at, int64_t total, int grid) {
  const int64_t c = sharers(total, grid), x = (at + 1) * c - 1;
  // (a division of 64 bits takes five times as long, and every row needs four)
  if ((total * c) >> 32 == 0)
    return static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(total));
  return static_cast<int>(x / total);
}

// ------------------------------------------------------------------ tiles into shared memory
// A ring of R slots, each one tile of keys or of values. Keys and values have
// rings of their own, since a tile of values is held until its probabilities are
// known. bf16 operands: 128-byte swizzle, boxes of 128 tokens x 64 channels. E4M3
// keys are operands as they are (8-bit products): 128 tokens of D bytes, swizzled
// by D bytes; the queries are then two codes a value, so that no bit of theirs is
// lost. E4M3 values become bf16 first, since P has the range of bf16.
template <int R>
struct RingBars {
  uint64_t full[R], empty[R];
};

// A page of a sequence; one outside the pool is reported, and page 0 read in its place.
__device__ __forceinline__ int checked_page(const PoolView& v, int seq, int j) {
  const int p = v.table[static_cast<size_t>(seq) * v.width + j];
  if (p >= 0 && p < v.pages) return p;
  atomicOr(v.err, kErrBadState);
  return 0;
}

// ONCE: the call reads the page only here, so that its lines need not displace the
// logits and pieces in L2, which are read again (16 rows of 32768 keys x 32 heads: 160 -> 151.5
// us, 256 sequences 290 -> 280.5).
template <bool ONCE>
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar) {
  if constexpr (ONCE)
    tma_load_2d_once(dst, map, c0, c1, bar);
  else
    tma_load_2d(dst, map, c0, c1, bar);
}

// bf16 pool, one warp: lane i fetches the boxes of page i of a tile by TMA;
// pages behind the last token are left out, so rows of the slot behind it hold
// anything. Cursor: step() moves to the next tile (false: none), with seq, len, h, kt.
template <int D, bool ONCE, int R, typename Cursor>
__device__ void produce_tma(const PoolView& v, const CUtensorMap* map, uint8_t* ring,
                            RingBars<R>& bars, Cursor c) {
  const int lane = threadIdx.x & 31, per = TILE_KEYS >> v.shift;
  uint32_t n = 0;
  for (; c.step(); ++n) {
    const int left = c.len - c.kt * TILE_KEYS, boxes = min(per, (left + v.page - 1) >> v.shift);
    const int row = lane < boxes
                        ? (checked_page(v, c.seq, c.kt * per + lane) * v.heads + c.h) << v.shift
                        : 0;
    const uint32_t st = n % R;
    if (n >= R && !pool_warp_wait(&bars.empty[st], ((n / R) - 1) & 1, v.err)) break;
    if (lane == 0) mbar_arrive_expect_tx(&bars.full[st], boxes * v.page * D * 2);
    __syncwarp();
    if (lane < boxes) {
#pragma unroll
      for (int b = 0; b < D / 64; ++b)
        load_box<ONCE>(ring + st * (TILE_KEYS * D * 2) + b * kBoxBytes + (lane << v.shift) * 128, map,
                       b * 64, row, &bars.full[st]);
    }
  }
  drain_copies(bars.full, n, v.err);
}

// Four E4M3 codes to bf16, exactly (three significant bits more than a code has).
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t w) {
  uint2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw hr =
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
    (i ? r.y : r.x) = pack_bf16x2(f.x, f.y);
  }
  return r;
}

// E4M3 pool, one warp: codes as they are, and their scales behind them in `scales`
// [R][128]. What lies behind the last token holds anything.
template <int D, bool ONCE, int R, typename Cursor>
__device__ void produce_codes(const PoolView& v, const CUtensorMap* map, const float* scale,
                              uint8_t* ring, float* scales, RingBars<R>& bars, Cursor c) {
  const int lane = threadIdx.x & 31, per = TILE_KEYS >> v.shift;
  uint32_t n = 0;
  for (; c.step(); ++n) {
    const int left = c.len - c.kt * TILE_KEYS, boxes = min(per, (left + v.page - 1) >> v.shift);
    const int row = lane < boxes
                        ? (checked_page(v, c.seq, c.kt * per + lane) * v.heads + c.h) << v.shift
                        : 0;
    const uint32_t st = n % R;
    if (n >= R && !pool_warp_wait(&bars.empty[st], ((n / R) - 1) & 1, v.err)) break;
    if (lane == 0) mbar_arrive_expect_tx(&bars.full[st], boxes * v.page * (D + 4));
    __syncwarp();
    if (lane < boxes) {
      load_box<ONCE>(ring + st * (TILE_KEYS * D) + (lane << v.shift) * D, map, 0, row, &bars.full[st]);
      bulk_copy_g2s(scales + st * TILE_KEYS + (lane << v.shift), scale + row, v.page * 4, &bars.full[st]);
    }
  }
  drain_copies(bars.full, n, v.err);
}

// The two bf16 terms of a probability: its upper 16 bits as they are, and what is left, rounded
// (the terms' sum is off by 2^-16 of p at most). For bf16 values the lowest bit is set first, so
// that the second term of a p that has a first one is above zero: an infinite value stays one in
// both products, where 0 would make a NaN of it. (Codes have no infinity.)
template <bool F8>
__device__ __forceinline__ uint32_t split_bits(float p) {
  return __float_as_uint(p) | (F8 ? 0u : 1u);
}
__device__ __forceinline__ float split_first(uint32_t bits) { return __uint_as_float(bits & 0xffff0000u); }

// E4M3 pool, NT threads: tiles of value codes (linear, S slots) to bf16 operands,
// and their scales to out_scales [kScaleTiles][128] by tile; rows behind the last
// token become zero. Each warp arrives once on a slot's barriers. (Codes loaded
// through registers of the converting threads took 10,000 clocks a tile of keys
// and values: every use of one load waited for all of them.)
constexpr int kScaleTiles = 8;  // more tiles than lie between a conversion and its reader

template <int D, int R, int S, int NT, typename Cursor>
__device__ void convert_values(const PoolView& v, const uint8_t* codes, const float* scales,
                               RingBars<S>& from, uint8_t* ring, RingBars<R>& to,
                               float* out_scales, Cursor c, int tid) {
  constexpr int CPR = D / 16;               // 16-byte chunks of codes per token
  constexpr int NCH = TILE_KEYS * CPR / NT;  // chunks per thread and slot
  const int lane = threadIdx.x & 31;
  for (uint32_t n = 0; c.step(); ++n) {
    const int valid = c.len - c.kt * TILE_KEYS;
    const uint32_t sc = n % S, st = n % R;
    if (!pool_warp_wait(&from.full[sc], (n / S) & 1, v.err)) return;
    const uint4* src = reinterpret_cast<const uint4*>(codes + sc * (TILE_KEYS * D));
    uint4 x[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      x[i] = src[tid + NT * i];
      if ((tid + NT * i) / CPR >= valid) x[i] = make_uint4(0, 0, 0, 0);
    }
    float scale = 0.f;
    if (tid < TILE_KEYS && tid < valid) scale = scales[sc * TILE_KEYS + tid];
    if (n >= R && !pool_warp_wait(&to.empty[st], ((n / R) - 1) & 1, v.err)) return;
    if (tid < TILE_KEYS) out_scales[(n % kScaleTiles) * TILE_KEYS + tid] = scale;
    uint8_t* dst = ring + st * (TILE_KEYS * D * 2);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int q = tid + NT * i, row = q / CPR, col = q % CPR;
      const uint2 a = e4m3x4_to_bf16(x[i].x), b = e4m3x4_to_bf16(x[i].y);
      const uint2 e = e4m3x4_to_bf16(x[i].z), f = e4m3x4_to_bf16(x[i].w);
      uint8_t* at = dst + (col >> 2) * kBoxBytes + row * 128;
      const int c0 = 2 * (col & 3);
      // the two boxes of a row lie in the same banks: the halves of a row write
      // their even and odd chunks in opposite order
      const bool swap = col >= 4;
      const uint4 even = make_uint4(a.x, a.y, b.x, b.y), odd = make_uint4(e.x, e.y, f.x, f.y);
      *reinterpret_cast<uint4*>(at + (((c0 + swap) ^ (row & 7)) << 4)) = swap ? odd : even;
      *reinterpret_cast<uint4*>(at + (((c0 + !swap) ^ (row & 7)) << 4)) = swap ? even : odd;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&to.full[st]);
      mbar_arrive(&from.empty[sc]);
    }
  }
}

// K-major E4M3 operand with rows of D bytes: k-step kk is 32 bytes further.
template <int D>
__device__ __forceinline__ uint64_t desc_codes(const uint8_t* tile) {
  return D == 128 ? smem_desc(tile, 16, 1024) : smem_desc_64(tile, 16, 512);
}
// ------------------------------------------------------------------ records
// Where the records of a (entry, key head) unit's rows are: `prefix` of the
// prefix, then `own` of the own tokens. Record i of row g is at base + i * step + g.
struct Records {
  int prefix, own;
  size_t pbase, pstep, obase;
};

// owners(at, total, c): the CTAs c[4] that had tiles at[4] of lists of total[2] tiles:
// the first and last tile of the prefix unit that holds the rows (list 0), then
// of the own unit (list 1). cum: own tiles before the entry, before the next, of all.
template <typename Owners>
__device__ __forceinline__ Records place_records(const AttendParams& p, int b, int h, int plen,
                                                 const int (&cum)[3], Owners&& owners) {
  Records x{};
  const int pt = p.a.prefix >= 0 ? key_tiles(plen) : 0, tiles = cum[1] - cum[0];
  const int64_t own = static_cast<int64_t>(cum[2]) * p.s.heads;
  const int64_t pre = static_cast<int64_t>(p.s.heads) * (p.s.few ? 1 : p.s.blocks) * pt;
  const int64_t ototal = own + (p.s.few ? pre : 0), ptotal = p.s.few ? ototal : pre;
  const int qt = b / p.s.per_tile, r0 = (b - qt * p.s.per_tile) * p.s.group;
  const int u = p.s.few ? h : h * p.s.blocks + (qt >> 1);
  const int64_t pa = static_cast<int64_t>(u) * pt;
  const int64_t oa = (p.s.few ? pre : 0) + static_cast<int64_t>(cum[0]) * p.s.heads +
                     static_cast<int64_t>(h) * tiles;
  int c[4];
  owners({pa, pa + pt - 1, oa, oa + tiles - 1}, {ptotal, ototal}, c);
  if (pt) {
    x.prefix = c[1] - c[0] + 1;
    const size_t piece = u + c[0];
    if (p.s.few) {
      x.pbase = piece * kFewRows + r0;
      x.pstep = kFewRows;
    } else if ((qt | 1) < p.s.nq) {  // a block of two row tiles: a record per tile
      x.pbase = (piece * 2 + (qt & 1)) * TILE_ROWS + r0;
      x.pstep = 2 * TILE_ROWS;
    } else {                         // one row tile: a record per half of the keys
      x.pbase = piece * 2 * TILE_ROWS + r0;
      x.pstep = TILE_ROWS;
      x.prefix *= 2;
    }
  }
  if (tiles) {
    x.own = c[3] - c[2] + 1;
    x.obase = static_cast<size_t>(b * p.s.heads + h + c[2]) * p.s.group;
  }
  return x;
}

// Index of record i of row g in its array (the prefix's for i < x.prefix), and its {max, sum}.
__device__ __forceinline__ size_t record(const AttendParams& p, const Records& x, int i, int g) {
  return (i < x.prefix ? x.pbase + i * x.pstep
                       : x.obase + static_cast<size_t>(i - x.prefix) * p.s.group) + g;
}
template <bool L2 = false>
__device__ __forceinline__ float2 record_ml(const AttendParams& p, const Records& x, int i, int g) {
  return load<L2>((i < x.prefix ? p.w.pml : p.w.tml) + record(p, x, i, g));
}

// Adds a record to {m, l}.
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2);
  if (top != -INFINITY)
    l = l * ex2(m - top) + l2 * ex2(m2 - top);
  else
    l += l2;  // a NaN sum stays one
  m = top;
}
#endif  // __CUDACC__

}  // namespace h2o
