// Shared parts of the paged attention kernels: the scratch of a call, the list
// of 128-key tiles that CTAs share, and the producers that bring tiles of keys
// and values into shared memory as bf16 matrix operands.
#pragma once

#include "common.cuh"
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
// Tensor maps (pool_attend.cu): queries [n][heads][group][d] in boxes of
// `entries` groups of one head x 64 channels; a pool's keys or values in boxes of
// a page's tokens x 64 channels (bf16, 128-byte swizzle) or x all codes (E4M3).
cudaError_t query_map(CUtensorMap* m, const AttendArgs& a, int entries);
cudaError_t page_map(CUtensorMap* m, const void* base, const PoolView& v);

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

#ifdef __CUDACC__
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
// A ring of R slots, each one tile of keys or values as bf16, 128-byte swizzled:
// boxes of 128 tokens x 64 channels. Slots are filled in the order K, V, K, V,
// ... of a cursor's tiles (K only where values are not wanted).
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
template <int D, int R, bool VALUES, typename Cursor>
__device__ void produce_tma(const PoolView& v, const CUtensorMap* tk, const CUtensorMap* tv,
                            uint8_t* ring, RingBars<R>& bars, Cursor c) {
  constexpr int BYTES = TILE_KEYS * D * 2;
  const int lane = threadIdx.x & 31, per = TILE_KEYS >> v.shift;
  uint32_t n = 0;
  while (c.step()) {
    const int left = c.len - c.kt * TILE_KEYS, boxes = min(per, (left + v.page - 1) >> v.shift);
    const int row = lane < boxes
                        ? (checked_page(v, c.seq, c.kt * per + lane) * v.heads + c.h) << v.shift
                        : 0;
#pragma unroll
    for (int kv = 0; kv < (VALUES ? 2 : 1); ++kv, ++n) {
      const uint32_t st = n % R;
      if (n >= R && !warp_wait(&bars.empty[st], ((n / R) - 1) & 1, v.err)) return;
      if (lane == 0) mbar_arrive_expect_tx(&bars.full[st], boxes * v.page * D * 2);
      __syncwarp();
      if (lane < boxes) {
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
          tma_load_2d(ring + st * BYTES + b * kBoxBytes + (lane << v.shift) * 128, kv ? tv : tk,
                      b * 64, row, &bars.full[st]);
      }
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

// E4M3 pool: a second ring of S slots takes the codes as they are (128 tokens of
// D bytes, then 128 scales), by TMA from one warp, like produce_tma; NT other
// threads turn each into a slot of bf16. (Codes loaded through registers of the
// converting threads, three slots ahead, took 10,000 clocks a tile of keys and
// values against 2,500 this way: every use of one load waited for all of them.)
template <int S>
struct CodeBars {
  uint64_t full[S], empty[S];  // empty: an arrival per converting warp
};

template <int D>
constexpr int kCodeSlot = TILE_KEYS * D + TILE_KEYS * 4;

template <int D, int S, bool VALUES, typename Cursor>
__device__ void fetch_codes(const PoolView& v, const CUtensorMap* tk, const CUtensorMap* tv,
                            uint8_t* codes, CodeBars<S>& bars, Cursor c) {
  const int lane = threadIdx.x & 31, per = TILE_KEYS >> v.shift;
  uint32_t n = 0;
  while (c.step()) {
    const int left = c.len - c.kt * TILE_KEYS, boxes = min(per, (left + v.page - 1) >> v.shift);
    const int row = lane < boxes
                        ? (checked_page(v, c.seq, c.kt * per + lane) * v.heads + c.h) << v.shift
                        : 0;
#pragma unroll
    for (int kv = 0; kv < (VALUES ? 2 : 1); ++kv, ++n) {
      const uint32_t st = n % S;
      if (n >= S && !warp_wait(&bars.empty[st], ((n / S) - 1) & 1, v.err)) return;
      if (lane == 0) mbar_arrive_expect_tx(&bars.full[st], boxes * v.page * (D + 4));
      __syncwarp();
      if (lane < boxes) {
        uint8_t* dst = codes + st * kCodeSlot<D>;
        tma_load_2d(dst + (lane << v.shift) * D, kv ? tv : tk, 0, row, &bars.full[st]);
        bulk_copy_g2s(dst + TILE_KEYS * D + (lane << v.shift) * 4, (kv ? v.vscale : v.kscale) + row,
                      v.page * 4, &bars.full[st]);
      }
    }
  }
}

// Rows behind the last token become zero. The scales of tile g go to
// scales[g % kScaleTiles<VALUES>][0: keys, 1: values][128]. Each warp arrives once
// on the slot's barrier.
template <int D, int R, int S, bool VALUES, int NT, typename Cursor>
__device__ void convert_codes(const PoolView& v, const uint8_t* codes, CodeBars<S>& from,
                              uint8_t* ring, RingBars<R>& to, float* scales, Cursor c, int tid) {
  constexpr int BYTES = TILE_KEYS * D * 2;
  constexpr int CPR = D / 16;               // 16-byte chunks of codes per token
  constexpr int NCH = TILE_KEYS * CPR / NT;  // chunks per thread and slot
  const int lane = threadIdx.x & 31;
  uint32_t n = 0;
  while (c.step()) {
    const int valid = c.len - c.kt * TILE_KEYS;
#pragma unroll
    for (int kv = 0; kv < (VALUES ? 2 : 1); ++kv, ++n) {
      const uint32_t sc = n % S, st = n % R;
      if (!warp_wait(&from.full[sc], (n / S) & 1, v.err)) return;
      const uint8_t* src = codes + sc * kCodeSlot<D>;
      uint4 x[NCH];
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        x[i] = reinterpret_cast<const uint4*>(src)[tid + NT * i];
        if ((tid + NT * i) / CPR >= valid) x[i] = make_uint4(0, 0, 0, 0);
      }
      if (tid < TILE_KEYS)
        scales[(((VALUES ? n >> 1 : n) % kScaleTiles<VALUES>) * 2 + kv) * TILE_KEYS + tid] =
            tid < valid ? reinterpret_cast<const float*>(src + TILE_KEYS * D)[tid] : 0.f;
      if (n >= R && !warp_wait(&to.empty[st], ((n / R) - 1) & 1, v.err)) return;
      uint8_t* dst = ring + st * BYTES;
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
}
#endif  // __CUDACC__

}  // namespace h2o
