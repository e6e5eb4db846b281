// What the accepted drafts of a batch attended to: for every accepted row (its query
// q and the lse that attention left) and every token j that it sees, the score of j
// grows by p_j = exp(q . k_j / sqrt(d) - lse), summed over the rows of a head's query
// group: what single-token attention would have added, had the drafts been decoded
// one by one.
//
// Bound: keys are read once, 2 d bytes a token and head (d + 4 in E4M3), against 2 d
// flops a row; a sequence keeps few drafts, so the bytes decide. A CTA goes through its
// share of the 128-key tiles; a warp has 16 keys of a tile and copies them, whole rows,
// into its part of a ring of shared memory while it works on the tile before. They are
// operands of mma (m16 n8 k16: keys are the long side, the rows eight at a time): the
// channels of a lane's 16-byte read are taken for those of its places in two products,
// and the queries' for the same, since a dot product does not mind their order. Rows lie
// in shared memory, 64 at a time, and the next 64 (or the next tile's, where they are
// others) are on their way beside the products; the prefix's are those of all sequences, as
// one list. Sums are fp32 in the order of the rows.
//
// Measured in a graph, with the fork, the drafts' write and the other kernels of accept: four
// documents of 32768 tokens, 32 heads of bf16 (1.07 GB) 211 us; 64 sequences of up to 2000
// tokens, 8 heads of E4M3 (85 MB) 65 us (calls back to back 73), under a prefix of 8197 168 (rows
// staged when they are needed: 64.5 and 270). Before: one chain of products for a row's sum, and the mask
// tested at every logit 66.5; keys loaded straight into registers, four blocks an SM, 216
// and 72; 32 keys a warp 248; a lane's own 64-byte pieces of rows through the ring 217 and
// 68; the next tile in registers 260 and 77. One block an SM took 277 and 94.
#include <type_traits>

#include "common.cuh"
#include "device_state.h"
#include "kernels.h"
#include "pool_tiles.cuh"

namespace h2o {
namespace {

constexpr int kThreads = 256, kRows = 64;
constexpr int kM = kScoreKeys / (kThreads / 32) / 16;  // products of 16 keys a warp
constexpr int kStages = 2, kBlocks = 2;                // tiles in the ring; blocks of an SM

// Bytes of the keys on their way: rows, then (E4M3) their scales.
template <int D, bool F8>
constexpr int ring_bytes() {
  return kStages * kScoreKeys * (F8 ? D + 4 : 2 * D);
}

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four E4M3 codes times 2^-11 to bf16, exactly (the smallest code is then 2^-20, and halves go down to
// 2^-24). A sum of d codes up to 448 times a query beyond 2^112 would leave fp32 although the logit, with
// the key's scale, does not; so the sum stays inside up to 2^123, where a key of 2^-119, the least that is
// stored, has logits of some 128. The key's scale is multiplied by 2^11 instead, with the softmax's factor by
// 2^8.6 at most, which the largest, 2^119.2, bears. (The batch of E4M3 above 63.6 -> 64.7 us; codes moved
// into bf16's places by bits, and one product, 67.)
constexpr float kCodeScale = 0x1p11f;
__device__ __forceinline__ uint2 small_codes(uint32_t w) {
  uint2 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__hmul2(*reinterpret_cast<const __half2*>(&hr), __float2half2_rn(1.f / kCodeScale)));
    (i ? r.y : r.x) = pack_bf16x2(f.x, f.y);
  }
  return r;
}

// Last i in [0, n) with cum[i] <= x.
__device__ __forceinline__ int last_at(const int32_t* cum, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads, kBlocks)
    accept_score_kernel(const __grid_constant__ AcceptArgs a, float qscale) {
  constexpr int CH = D / 8;                       // 16-byte chunks of a row
  constexpr int LD = F8 ? D / 64 : D / 32;        // loads of a lane and key
  __shared__ uint4 s_q[2][kRows * CH];            // rows in use, and the next
  __shared__ float s_lse[2][kRows];               // infinite: not counted
  __shared__ int s_first[2][kRows];               // accepted drafts before the row's own
  const PoolView& v = a.v;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  grid_dependency_wait();
  grid_launch_dependents();
  const int plen = a.prefix >= 0 ? max(0, checked_length(v, a.prefix, blockIdx.x + tid == 0)) : 0;
  const int all_rows = a.rows[a.n];
  const int ptiles = all_rows ? (plen + kScoreKeys - 1) / kScoreKeys : 0;
  const int64_t pre = static_cast<int64_t>(ptiles) * v.heads, own = static_cast<int64_t>(a.tiles[a.n]) * v.heads;

  // The CTA's tiles: its share of the prefix's, then of the sequences' own.
  struct Tile {
    int e, h, kt, tiles;      // entry (-1: the prefix), head, tile of a head's
    int seq, len, base, rows;  // tokens, those before the accepted drafts; rows
  };
  const int grid = gridDim.x, cta = blockIdx.x;
  const int64_t pre0 = share_begin(pre, grid, cta), own0 = share_begin(own, grid, cta);
  const int npre = static_cast<int>(share_begin(pre, grid, cta + 1) - pre0);
  const int count = npre + static_cast<int>(share_begin(own, grid, cta + 1) - own0);
  auto enter = [&](Tile& x) {
    const int kept = a.plan[static_cast<size_t>(x.e) * kAcceptInts];
    x.tiles = a.tiles[x.e + 1] - a.tiles[x.e];
    x.seq = a.seqs[x.e];
    x.base = a.plan[static_cast<size_t>(x.e) * kAcceptInts + 1];
    x.len = x.base + kept;
    x.rows = kept * a.group;
  };
  // tile i of the share, from the one before it
  auto step = [&](Tile& x, int i) {
    if (i == npre) {
      x.e = last_at(a.tiles, a.n, static_cast<int>(own0 / v.heads));
      enter(x);
      const int k = static_cast<int>(own0 - static_cast<int64_t>(a.tiles[x.e]) * v.heads);
      x.h = k / x.tiles;
      x.kt = k - x.h * x.tiles;
    } else if (i == 0) {
      x.h = static_cast<int>(pre0 / ptiles);
      x.kt = static_cast<int>(pre0 - static_cast<int64_t>(x.h) * ptiles);
      x.e = -1;
      x.tiles = ptiles;
      x.seq = a.prefix;
      x.len = x.base = plen;
      x.rows = all_rows * a.group;
    } else if (++x.kt == x.tiles) {
      x.kt = 0;
      if (++x.h == v.heads) {
        x.h = 0;
        do ++x.e;
        while (a.tiles[x.e + 1] == a.tiles[x.e]);
        enter(x);
      }
    }
  };
  // This warp's keys of tile i, 16 of them with one page: a row after the other, 512 bytes a
  // load. A row's 16-byte chunks are exchanged by its number, so that the lanes that read the same
  // chunk of eight rows meet different banks. Rows behind a sequence's last lie in its page.
  constexpr int CK = F8 ? D / 16 : D / 8;         // chunks of a key
  constexpr int kWarpKeys = 16 * kM;
  extern __shared__ __align__(16) uint8_t ring[];
  uint4* const s_k = reinterpret_cast<uint4*>(ring) + warp * kStages * kWarpKeys * CK;
  float* const s_ks =
      reinterpret_cast<float*>(ring + kStages * kScoreKeys * CK * 16) + warp * kStages * kWarpKeys;
  Tile ahead = {}, x = {};
  auto fetch = [&](int i) {
    if (i < count) {
      step(ahead, i);
      const int k0 = ahead.kt * kScoreKeys + warp * kWarpKeys, at = i % kStages * kWarpKeys;
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const int key = k0 + 16 * m;
        if (key < ahead.len) {
          const int p = checked_page(v, ahead.seq, key >> v.shift);
          const size_t slot = ((static_cast<size_t>(p) * v.heads + ahead.h) << v.shift) + (key & (v.page - 1));
          const uint4* src = reinterpret_cast<const uint4*>(v.K + slot * v.row_bytes) + lane;
#pragma unroll
          for (int y = 0; y < CK / 2; ++y) {
            const int r = (y * 32 + lane) / CK, ch = lane % CK;
            copy_async(s_k + (at + 16 * m + r) * CK + (ch ^ (CK < 8 ? 0 : (r & 1) * 4)), src + y * 32);
          }
          if (F8 && lane < 4) copy_async(s_ks + at + 16 * m + 4 * lane, v.kscale + slot + 4 * lane);
        }
      }
    }
    copy_async_commit();
  };
  // A tile's rows from r0 on, to buffer `to`, as one more group of copies.
  auto stage = [&](const Tile& of, int r0, int to) {
    const int32_t* list = a.list + (of.e < 0 ? 0 : a.rows[of.e]);
#pragma unroll
    for (int y = tid; y < kRows * CH; y += kThreads) {
      const int r = y / CH, ch = y % CH, at = r0 + r;
      if (at < of.rows) {
        const int i = at / a.group;
        const size_t row = static_cast<size_t>(list[i]) * (v.heads * a.group) + of.h * a.group + (at - i * a.group);
        copy_async(&s_q[to][r * CH + (ch ^ (F8 ? r & 1 : (r & 1) * 4))], static_cast<const uint4*>(a.q) + row * CH + ch);
        if (ch == 0) {
          copy_async_4(&s_lse[to][r], a.lse + row);
          s_first[to][r] = i;
        }
      } else if (ch == 0) {
        s_lse[to][r] = INFINITY;
        s_first[to][r] = 0;
      }
    }
    copy_async_commit();
  };

  // Buffer `rows` is in use; `staged`: the other has what comes next, or will have.
  int rows = 1;
  bool staged = count > 0;
  fetch(0);
  if (staged) stage(ahead, 0, 0);
  for (int i = 0; i < count; ++i) {
    __syncwarp();
    fetch(i + 1);
    copy_async_wait<1>();  // all but what was just asked for
    __syncwarp();
    step(x, i);
    uint32_t k[kM][2][D / 8];  // of a key: this lane's channels, in pairs
    float ks[kM][2], sum[kM][2];
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = 8 * u + g, at = i % kStages * kWarpKeys + 16 * m + r;
        sum[m][u] = 0.f;
        ks[m][u] = F8 ? s_ks[at] * (kCodeScale * qscale) : qscale;
#pragma unroll
        for (int y = 0; y < LD; ++y) {
          const uint4 raw = s_k[at * CK + ((4 * y + c) ^ (CK < 8 ? 0 : (r & 1) * 4))];
          const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            if constexpr (F8) {
              const uint2 pair = small_codes(w[z]);
              k[m][u][8 * y + 2 * z] = pair.x;
              k[m][u][8 * y + 2 * z + 1] = pair.y;
            } else {
              k[m][u][4 * y + z] = w[z];
            }
          }
        }
      }
    const int k0 = x.kt * kScoreKeys + warp * 16 * kM;
    float* const score = v.score + (static_cast<size_t>(x.seq) * v.heads + x.h) * v.cap;
    float old[kM][2];
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int key = k0 + 16 * m + 8 * u + g;
        old[m][u] = c == 0 && key < x.len ? score[key] : 0.f;
      }
    for (int r0 = 0; r0 < x.rows; r0 += kRows) {
      if (staged) {
        if (r0) copy_async_wait<0>();
        __syncthreads();
        rows ^= 1;
      }
      staged = true;
      if (r0 + kRows < x.rows)
        stage(x, r0 + kRows, rows ^ 1);
      else if (i + 1 < count && (ahead.rows > kRows || ahead.h != x.h || ahead.e != x.e))
        stage(ahead, 0, rows ^ 1);
      else
        staged = false;
      const int live = min(kRows, x.rows - r0);
      // drafts among this warp's keys, which the rows before them do not see
      const bool masked = x.e >= 0 && k0 + 16 * kM > x.base;
      auto rows8 = [&](auto drafts_too, int t) {
        constexpr bool M = decltype(drafts_too)::value;
        float acc[kM][4] = {}, acc2[kM][4] = {};  // (two chains, each half as long)
        const int r = t + g;
        const uint4* q = s_q[rows] + r * CH;
#pragma unroll
        for (int y = 0; y < CH / 4; ++y) {
          // chunks of a row in the lane's order: bf16 4 y + c; E4M3 8 (y / 2) + 2 c + y % 2
          const int ch = F8 ? 8 * (y / 2) + 2 * c + y % 2 : 4 * y + c;
          const uint4 b = q[ch ^ (F8 ? r & 1 : (r & 1) * 4)];
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            mma_16x8x16(acc[m], k[m][0][4 * y], k[m][1][4 * y], k[m][0][4 * y + 1], k[m][1][4 * y + 1], b.x, b.y);
            mma_16x8x16(acc2[m], k[m][0][4 * y + 2], k[m][1][4 * y + 2], k[m][0][4 * y + 3], k[m][1][4 * y + 3], b.z,
                        b.w);
          }
        }
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int z = 0; z < 4; ++z) acc[m][z] += acc2[m][z];
        // column 2 c + z of the eight rows
        const float2 l = *reinterpret_cast<const float2*>(s_lse[rows] + t + 2 * c);
        const int2 f = *reinterpret_cast<const int2*>(s_first[rows] + t + 2 * c);
        const float2 n = make_float2(fabsf(l.x) == INFINITY ? INFINITY : l.x * kLog2e,
                                     fabsf(l.y) == INFINITY ? INFINITY : l.y * kLog2e);
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int draft = k0 + 16 * m + 8 * u + g - x.base;  // below 0: none
            const float p0 = ex2(fmaf(acc[m][2 * u], ks[m][u], -n.x)), p1 = ex2(fmaf(acc[m][2 * u + 1], ks[m][u], -n.y));
            sum[m][u] += n.x == INFINITY || (M && draft > f.x) ? 0.f : p0;
            sum[m][u] += n.y == INFINITY || (M && draft > f.y) ? 0.f : p1;
          }
      };
      if (masked)
        for (int t = 0; t < live; t += 8) rows8(std::true_type{}, t);
      else
        for (int t = 0; t < live; t += 8) rows8(std::false_type{}, t);
    }
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float y = sum[m][u];
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        y += __shfl_xor_sync(0xffffffffu, y, 2);
        const int key = k0 + 16 * m + 8 * u + g;
        if (c == 0 && key < x.len) score[key] = old[m][u] + y;
      }
  }
  copy_async_wait<0>();
}

template <int D, bool F8>
cudaError_t launch(const AcceptArgs& a, cudaStream_t stream) {
  static int opted_in[kMaxDevices] = {};
  constexpr int smem = ring_bytes<D, F8>();
  const auto kern = accept_score_kernel<D, F8>;
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(kern), smem, opted_in);
  if (e != cudaSuccess) return e;
  const float qscale = kLog2e / sqrtf(static_cast<float>(D));
  return launch_after(kern, dim3(kBlocks * num_sms()), kThreads, smem, stream, a, qscale);
}

}  // namespace

cudaError_t pool_accept_scores(const AcceptArgs& a, cudaStream_t stream) {
  if (a.v.kscale) return a.v.d == 128 ? launch<128, true>(a, stream) : launch<64, true>(a, stream);
  return a.v.d == 128 ? launch<128, false>(a, stream) : launch<64, false>(a, stream);
}

}  // namespace h2o
