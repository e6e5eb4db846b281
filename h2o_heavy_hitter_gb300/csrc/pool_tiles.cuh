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
  bool few;      // the prefix has at most kFewRows query rows per head
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
  float* nlse;     // [heads][nq][128] -lse (base 2) of a prefix row, -inf: not counted (accumulate only)
  float2* pml;     // prefix pieces {max, sum}: many rows [heads * blocks + grid][2][128],
                   // few rows [heads + grid][kFewRows]
  float2* tml;     // own pieces [n * heads + grid][group]
  float* po;       // prefix pieces' outputs, [d] per row
  float* to;       // own pieces' outputs
  float* logits;   // [n][heads][group][cap] base-2 logits of the own tokens (accumulate only)
  float* plogits;  // [heads][n * group][cap] of the prefix (accumulate, few rows only)
};

struct AttendParams {
  AttendArgs a;
  Shape s;
  AttendScratch w;
  float qscale;  // log2(e) / sqrt(d)
};

// Launchers of the kernels for a prefix with many rows (pool_prefix.cu). The
// first leaves pieces, the second adds the prefix's scores.
cudaError_t pool_prefix(const AttendParams& p, cudaStream_t stream);
cudaError_t pool_prefix_score(const AttendParams& p, cudaStream_t stream);
// Tensor map of the queries [n][heads][group][d] in boxes of `entries` groups of
// one head x 64 channels (pool_attend.cu).
cudaError_t query_map(CUtensorMap* m, const AttendArgs& a, int entries);

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
// The result is made warp-uniform (see warp_wait).
__device__ __forceinline__ bool pool_warp_wait(uint64_t* bar, uint32_t parity, int32_t* err) {
  return __all_sync(0xffffffffu, pool_wait(bar, parity, err));
}

// ------------------------------------------------------------------ lengths, shares
// A sequence's length, -1 (reported when `report`) for a state that no call leaves.
__device__ __forceinline__ int checked_length(const PoolView& v, int seq, bool report) {
  const int len = v.meta[2 * seq];
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
  return static_cast<int>(((at + 1) * sharers(total, grid) - 1) / total);
}

// ------------------------------------------------------------------ tiles into shared memory
// A ring of R slots, each one tile of keys or of values as bf16, 128-byte
// swizzled: boxes of 128 tokens x 64 channels. Keys and values have rings of their
// own, since a tile of values is held until its probabilities are known.
template <int R>
struct RingBars {
  uint64_t full[R], empty[R];
};

// Tiles whose scales are kept: more than can be between a slot's refill and the
// reader of its scales (a value tile is held until its reader is done, a key
// tile only until its product is).
template <bool VALUES>
constexpr int kScaleTiles = VALUES ? 8 : 16;

// A page of a sequence; one outside the pool is reported, and page 0 read in its place.
__device__ __forceinline__ int checked_page(const PoolView& v, int seq, int j) {
  const int p = v.table[static_cast<size_t>(seq) * v.width + j];
  if (p >= 0 && p < v.pages) return p;
  atomicOr(v.err, kErrBadState);
  return 0;
}

// bf16 pool, one warp: lane i fetches the boxes of page i of a tile by TMA;
// pages behind the last token are left out, so rows of the slot behind it hold
// anything. Cursor: step() moves to the next tile (false: none), with seq, len, h, kt.
template <int D, int R, typename Cursor>
__device__ void produce_tma(const PoolView& v, const CUtensorMap* map, uint8_t* ring,
                            RingBars<R>& bars, Cursor c) {
  const int lane = threadIdx.x & 31, per = TILE_KEYS >> v.shift;
  for (uint32_t n = 0; c.step(); ++n) {
    const int left = c.len - c.kt * TILE_KEYS, boxes = min(per, (left + v.page - 1) >> v.shift);
    const int row = lane < boxes
                        ? (checked_page(v, c.seq, c.kt * per + lane) * v.heads + c.h) << v.shift
                        : 0;
    const uint32_t st = n % R;
    if (n >= R && !pool_warp_wait(&bars.empty[st], ((n / R) - 1) & 1, v.err)) return;
    if (lane == 0) mbar_arrive_expect_tx(&bars.full[st], boxes * v.page * D * 2);
    __syncwarp();
    if (lane < boxes) {
#pragma unroll
      for (int b = 0; b < D / 64; ++b)
        tma_load_2d(ring + st * (TILE_KEYS * D * 2) + b * kBoxBytes + (lane << v.shift) * 128, map,
                    b * 64, row, &bars.full[st]);
    }
  }
}

// Four E4M3 codes to bf16, exactly: the code's exponent and mantissa bits lie in
// the places of bf16's, with the exponent 120 too small.
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t w) {
  uint2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = __byte_perm(w, 0, i ? 0x3424 : 0x1404);
    const uint32_t t = ((x >> 4) & 0x07f007f0u) | (x & 0x80008000u);
    uint32_t y;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(t), "r"(0x7b807b80u));  // 2^120 twice
    (i ? r.y : r.x) = y;
  }
  return r;
}

// E4M3 pool: one more ring of S slots takes the codes as they are (128 tokens of
// D bytes, then 128 scales), by TMA from one warp; NT other threads turn each into
// a slot of bf16. Keys go one tile ahead of values (K0, K1, V0, K2, V1, ...), so
// that the next tile's keys are converted before the wait for this one's values'
// slot. (Codes loaded through registers of the converting threads took 10,000
// clocks a tile of keys and values: every use of one load waited for all of them.)
template <int S>
struct CodeBars {
  uint64_t full[S], empty[S];  // empty: an arrival per converting warp
  // Both scales of tile g are written: by g & 1, an arrival per converting warp.
  // (A reader may wait for it before the values of tile g - 1 are converted, but
  // never before those of g - 2: on the values' own barrier, whose phases may be
  // single tiles, that wait could take the phase before for its own.)
  uint64_t scaled[2];
};

template <int D>
constexpr int kCodeSlot = TILE_KEYS * D + TILE_KEYS * 4;

// The order of the code ring: calls f(tile, n, g, value) for the n-th slot, tile g.
// One call in one loop: the body is large, and several warps' bodies share the
// instruction cache.
struct CodeTile {
  int seq, len, h, kt;
};

template <bool VALUES, typename Cursor, typename F>
__device__ __forceinline__ void each_code_tile(Cursor keys, F&& f) {
  Cursor values = keys;
  uint32_t gk = 0, gv = 0;
  bool more = keys.step();
  for (uint32_t n = 0;; ++n) {
    const bool value = VALUES && (gk - gv == 2 || (!more && gk > gv));
    if (!value && !more) return;
    CodeTile c;
    if (value) {
      values.step();
      c = {values.seq, values.len, values.h, values.kt};
    } else {
      c = {keys.seq, keys.len, keys.h, keys.kt};
    }
    if (!f(c, n, value ? gv : gk, value)) return;
    if (value) {
      ++gv;
    } else {
      ++gk;
      more = keys.step();
    }
  }
}

template <int D, int S, bool VALUES, typename Cursor>
__device__ void fetch_codes(const PoolView& v, const CUtensorMap* tk, const CUtensorMap* tv,
                            uint8_t* codes, CodeBars<S>& bars, const Cursor& begin) {
  const int lane = threadIdx.x & 31, per = TILE_KEYS >> v.shift;
  each_code_tile<VALUES>(begin, [&](const CodeTile& c, uint32_t n, uint32_t, bool value) -> bool {
    const int left = c.len - c.kt * TILE_KEYS, boxes = min(per, (left + v.page - 1) >> v.shift);
    const int row = lane < boxes
                        ? (checked_page(v, c.seq, c.kt * per + lane) * v.heads + c.h) << v.shift
                        : 0;
    const uint32_t st = n % S;
    if (n >= S && !pool_warp_wait(&bars.empty[st], ((n / S) - 1) & 1, v.err)) return false;
    if (lane == 0) mbar_arrive_expect_tx(&bars.full[st], boxes * v.page * (D + 4));
    __syncwarp();
    if (lane < boxes) {
      uint8_t* dst = codes + st * kCodeSlot<D>;
      tma_load_2d(dst + (lane << v.shift) * D, value ? tv : tk, 0, row, &bars.full[st]);
      bulk_copy_g2s(dst + TILE_KEYS * D + (lane << v.shift) * 4, (value ? v.vscale : v.kscale) + row,
                    v.page * 4, &bars.full[st]);
    }
    return true;
  });
}

// Rows behind the last token become zero. The scales of tile g go to
// scales[g % kScaleTiles<VALUES>][0: keys, 1: values][128]. Each warp arrives once
// on the slot's barrier.
template <int D, int RK, int RV, int S, bool VALUES, int NT, typename Cursor>
__device__ void convert_codes(const PoolView& v, const uint8_t* codes, CodeBars<S>& from,
                              uint8_t* kring, RingBars<RK>& kbars, uint8_t* vring,
                              RingBars<RV>* vbars, float* scales, const Cursor& begin, int tid) {
  constexpr int BYTES = TILE_KEYS * D * 2;
  constexpr int CPR = D / 16;               // 16-byte chunks of codes per token
  constexpr int NCH = TILE_KEYS * CPR / NT;  // chunks per thread and slot
  const int lane = threadIdx.x & 31;
  each_code_tile<VALUES>(begin, [&](const CodeTile& c, uint32_t n, uint32_t g, bool value) -> bool {
    const int valid = c.len - c.kt * TILE_KEYS;
    const uint32_t sc = n % S;
    if (!pool_warp_wait(&from.full[sc], (n / S) & 1, v.err)) return false;
    const uint8_t* src = codes + sc * kCodeSlot<D>;
    uint4 x[NCH];
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      x[i] = reinterpret_cast<const uint4*>(src)[tid + NT * i];
      if ((tid + NT * i) / CPR >= valid) x[i] = make_uint4(0, 0, 0, 0);
    }
    float scale = 0.f;
    if (tid < TILE_KEYS && tid < valid) scale = reinterpret_cast<const float*>(src + TILE_KEYS * D)[tid];
    uint64_t* full;
    uint8_t* dst;
    if (VALUES && value) {
      if (g >= RV && !pool_warp_wait(&vbars->empty[g % RV], ((g / RV) - 1) & 1, v.err)) return false;
      full = &vbars->full[g % RV];
      dst = vring + g % RV * BYTES;
    } else {
      if (g >= RK && !pool_warp_wait(&kbars.empty[g % RK], ((g / RK) - 1) & 1, v.err)) return false;
      full = &kbars.full[g % RK];
      dst = kring + g % RK * BYTES;
    }
    if (tid < TILE_KEYS) scales[((g % kScaleTiles<VALUES>) * 2 + value) * TILE_KEYS + tid] = scale;
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
      mbar_arrive(full);
      mbar_arrive(&from.empty[sc]);
      if (VALUES && value) mbar_arrive(&from.scaled[g & 1]);
    }
    return true;
  });
}
#endif  // __CUDACC__

}  // namespace h2o
