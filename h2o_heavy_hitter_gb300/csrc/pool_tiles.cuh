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
// `entries` groups of one head x 64 channels; a bf16 pool's keys or values in
// boxes of a page's tokens x 64 channels.
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

// E4M3 pool, NT threads: codes from global memory through registers, PF slots
// ahead, into the slot as bf16; rows behind the last token become zero. The
// scales of tile g go to scales[g % kScaleTiles<VALUES>][0: keys, 1: values][128].
// Each warp arrives once on the slot's barrier.
template <int D, int R, bool VALUES, int NT, typename Cursor>
__device__ void produce_e4m3(const PoolView& v, uint8_t* ring, RingBars<R>& bars, float* scales,
                             Cursor c, int tid) {
  constexpr int BYTES = TILE_KEYS * D * 2;
  constexpr int CPR = D / 16;               // 16-byte chunks of codes per token
  constexpr int NCH = TILE_KEYS * CPR / NT;  // chunks per thread and slot
  constexpr int PF = NCH > 2 ? 3 : 4;  // what the registers of a 600-thread block hold
  const int lane = threadIdx.x & 31, per = TILE_KEYS >> v.shift;
  uint4 raw[PF][NCH];
  float sc[PF];
  bool live[PF];
  // The pages of the next tile are looked up while this one's tokens are on their
  // way: ahead, what `next` holds; then the slots (token, head) of this tile's rows.
  int next[NCH + 1];  // pages of this thread's rows, and of the row whose scale it loads
  int32_t slot[NCH + 1];
  auto row_of = [&](int i) { return i < NCH ? (tid + NT * i) / CPR : tid; };
  bool more = c.step();
  auto look_up = [&]() {
    const int valid = c.len - c.kt * TILE_KEYS;
    const int32_t* pages = v.table + static_cast<size_t>(c.seq) * v.width + c.kt * per;
#pragma unroll
    for (int i = 0; i <= NCH; ++i) {
      const int row = row_of(i);
      next[i] = row < TILE_KEYS && row < valid ? pages[row >> v.shift] : -1;
    }
  };
  if (more) look_up();
  bool value = false;  // the next slot to load
  auto load = [&](uint4 (&x)[NCH], float& s) -> bool {
    if (!VALUES || !value) {
      if (!more) return false;
      const int valid = c.len - c.kt * TILE_KEYS;
      bool bad = false;
#pragma unroll
      for (int i = 0; i <= NCH; ++i) {
        const int row = row_of(i);
        const bool in = row < TILE_KEYS && row < valid;
        const bool held = next[i] >= 0 && next[i] < v.pages;
        bad |= in && !held;
        slot[i] = in ? (((held ? next[i] : 0) * v.heads + c.h) << v.shift) + (row & (v.page - 1)) : -1;
      }
      if (bad) atomicOr(v.err, kErrBadState);  // page 0 is read in its place
      more = c.step();
      if (more) look_up();
    }
    const uint8_t* base = value ? v.V : v.K;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
      x[i] = slot[i] >= 0 ? *reinterpret_cast<const uint4*>(base + static_cast<size_t>(slot[i]) * D +
                                                             (tid + NT * i) % CPR * 16)
                          : make_uint4(0, 0, 0, 0);
    s = slot[NCH] >= 0 ? (value ? v.vscale : v.kscale)[slot[NCH]] : 0.f;
    if (VALUES) value = !value;
    return true;
  };
#pragma unroll
  for (int u = 0; u < PF; ++u) live[u] = load(raw[u], sc[u]);
  for (uint32_t n0 = 0;; n0 += PF) {
#pragma unroll
    for (int u = 0; u < PF; ++u) {
      if (!live[u]) return;
      const uint32_t n = n0 + u, st = n % R;
      if (n >= R && !warp_wait(&bars.empty[st], ((n / R) - 1) & 1, v.err)) return;
      uint8_t* dst = ring + st * BYTES;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int q = tid + NT * i, row = q / CPR, col = q % CPR;
        const uint2 a = e4m3x4_to_bf16(raw[u][i].x), b = e4m3x4_to_bf16(raw[u][i].y);
        const uint2 e = e4m3x4_to_bf16(raw[u][i].z), f = e4m3x4_to_bf16(raw[u][i].w);
        uint8_t* at = dst + (col >> 2) * kBoxBytes + row * 128;
        const int c0 = 2 * (col & 3);
        // the two boxes of a row lie in the same banks: the halves of a row write
        // their even and odd chunks in opposite order
        const bool swap = col >= 4;
        const uint4 even = make_uint4(a.x, a.y, b.x, b.y), odd = make_uint4(e.x, e.y, f.x, f.y);
        *reinterpret_cast<uint4*>(at + (((c0 + swap) ^ (row & 7)) << 4)) = swap ? odd : even;
        *reinterpret_cast<uint4*>(at + (((c0 + !swap) ^ (row & 7)) << 4)) = swap ? even : odd;
      }
      const uint32_t g = VALUES ? n >> 1 : n;
      if (tid < TILE_KEYS)
        scales[((g % kScaleTiles<VALUES>) * 2 + (VALUES ? n & 1 : 0)) * TILE_KEYS + tid] = sc[u];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.full[st]);
      live[u] = load(raw[u], sc[u]);
    }
  }
}
#endif  // __CUDACC__

}  // namespace h2o
