// Norms of queries and keys for each head with the rotation of their positions:
// from a projection's token-major output to head-major rows, or to the pages of a
// pool's sequences, whose positions only the device knows.
//
// For a head x of d channels: x <- x (mean x^2 + eps)^-1/2 w, then each pair (x, y)
// of the first `dim` channels becomes factor (x cos a - y sin a, x sin a + y cos a).
// The angle of pair i at position p is 2 pi frac(p turns_i / 2^64): the product
// wraps at whole turns, so it is exact for every p and the turns that there are (an fp32
// product p f is off by 0.06 rad at p = 2^20). Everything between the loads and the
// stores is fp32, each result rounded once.
//
// Bound by HBM, 4 bytes a channel: 32768 tokens of 3 x 32 heads of 128, 1.61 GB in 247
// us (6.5 TB/s); 8168 tokens of 48 heads with norms, 0.20 GB in 37.5 us; 8 prompts of up
// to 2048 tokens into a pool's pages, 0.70 GB in 121 us. D / 16 lanes own a head: a lane has the two
// 16-byte chunks whose channels are each other's pairs, in either layout, so that no
// channel changes lanes and only a norm's sum does. A warp takes one token's heads, 512 /
// D at a time: its lanes compute the token's cosines and sines once, two a lane, and
// hand them out by shuffles. Warps go from token to token without a barrier; each lane's
// own loads run kStages rounds ahead, into shared memory that no other lane reads.
#include <algorithm>

#include "common.cuh"
#include "device_state.h"
#include "rotary.h"
#include "tc.cuh"

namespace h2o {
namespace {

constexpr int kThreads = 256;
// Slots of a warp's ring, and blocks of an SM: the case of 32768 tokens took 296 us with 2 slots, 258
// with 4, and 306 with 3 blocks, whose 80 registers do not hold a head, its turns and its weights. (Loads
// into registers, two rounds at a time: 275 us, and 54 for the one with norms.)
constexpr int kStages = 3, kBlocks = 2;

struct Pages {
  PoolView v;
  const int32_t* seqs;
  const int32_t* plan;    // of pool_write_plan
  const int32_t* parent;  // or null
};

enum Sink { kRowsOut, kPagesBf16, kPagesF8 };

// Depth of node t below the first node of its branch, by one warp. A parent that is not an earlier
// node is reported and counts as none.
__device__ __forceinline__ int node_depth(const int32_t* parent, int T, int t, int32_t* err) {
  const int lane = threadIdx.x & 31;
  const int lo = lane < T ? parent[lane] : -1, hi = lane + 32 < T ? parent[lane + 32] : -1;
  int depth = 0;
  while (true) {
    const int a = __shfl_sync(0xffffffffu, lo, t & 31), b = __shfl_sync(0xffffffffu, hi, t & 31);
    const int p = t < 32 ? a : b;
    if (p < -1 || p >= t) {
      if (lane == 0) atomicOr(err, kErrBadList);
      return depth;
    }
    if (p < 0) return depth;
    t = p;
    ++depth;
  }
}

template <int D, Sink S>
__global__ void __launch_bounds__(kThreads, kBlocks)
    rotate_kernel(const __grid_constant__ RotateArgs a, const __grid_constant__ Pages p, int parts) {
  constexpr int LPR = D / 16, HEADS = 32 / LPR;  // lanes of a head, heads of a round
  constexpr int PPL = D / 64;                    // pairs whose angle a lane computes
  __shared__ uint4 s_ring[kThreads / 32][kStages * 64];
  const int lane = threadIdx.x & 31, l = lane % LPR, g = lane / LPR;
  const unsigned gmask = ((1u << LPR) - 1) << (g * LPR);
  // a token's rounds: the queries', then the keys', then the values'
  const int nq = (a.heads[0] + HEADS - 1) / HEADS, nk = nq + (a.heads[1] + HEADS - 1) / HEADS;
  const int rounds = nk + (a.heads[2] + HEADS - 1) / HEADS;
  const unsigned items = static_cast<unsigned>(a.n) * a.T * parts;  // (several parts only of few tokens)
  // This lane's chunks of eight channels: with pairs (i, i + dim / 2), chunks of pairs; else, and behind the
  // rotated channels, chunks that lie one behind the other over the lanes.
  const int rot = a.r.dim / 16;
  const int c0 = a.r.half && l >= rot ? l + rot : l, c1 = a.r.half && l < rot ? l + rot : l + LPR;
  const bool turn0 = a.r.half ? l < rot : l < 2 * rot, turn1 = a.r.half ? l < rot : l + LPR < 2 * rot;
  uint64_t turns[PPL];
#pragma unroll
  for (int i = 0; i < PPL; ++i) turns[i] = a.r.turns[lane * PPL + i];
  grid_dependency_wait();
  grid_launch_dependents();

  // the warp's rounds in order: every `stride`-th item, a part of a token's
  const unsigned stride = gridDim.x * (kThreads / 32);
  struct At {
    unsigned item;
    int token, e, t, i, last;
  };
  auto settle = [&](At& x) {  // at an item's first round, or at the first of the next that has any
    for (; x.item < items; x.item += stride) {
      x.token = x.item / parts;
      x.e = x.token / a.T;
      x.t = x.token - x.e * a.T;
      if (S != kRowsOut && x.t >= p.plan[x.e * kPlanInts]) continue;
      const int part = static_cast<int>(x.item) - x.token * parts;
      x.i = rounds * part / parts;
      x.last = rounds * (part + 1) / parts;
      break;
    }
  };
  At now, ahead;
  now.item = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  settle(now);
  ahead = now;
  // the loads' own position
  uint4* ring = s_ring[threadIdx.x / 32] + lane;
  const __nv_bfloat16* src = nullptr;
  int64_t further = 0;
  int left = 0;  // heads of the kind from this lane's on
  auto aim = [&] {
    const int kind = ahead.i < nq ? 0 : ahead.i < nk ? 1 : 2;
    const int h = (ahead.i - (kind == 0 ? 0 : kind == 1 ? nq : nk)) * HEADS + g;
    left = a.heads[kind] - h;
    further = HEADS * a.head[kind];
    src = static_cast<const __nv_bfloat16*>(a.in[kind]) + ahead.e * a.batch[kind] + ahead.t * a.token[kind] +
          h * a.head[kind];
  };
  auto fetch = [&](int st) {
    if (ahead.item < items) {
      if (left > 0) {
        copy_async(ring + st * 64, reinterpret_cast<const uint4*>(src) + c0);
        copy_async(ring + st * 64 + 32, reinterpret_cast<const uint4*>(src) + c1);
      }
      src += further;
      left -= HEADS;
      if (++ahead.i == ahead.last) {
        ahead.item += stride;
        settle(ahead);
        if (ahead.item < items) aim();
      } else if (ahead.i == nq || ahead.i == nk) {
        aim();
      }
    }
    copy_async_commit();
  };
  if (ahead.item < items) aim();
#pragma unroll
  for (int st = 0; st < kStages - 1; ++st) fetch(st);

  int st = 0;
  for (; now.item < items; now.item += stride, settle(now)) {
    const int e = now.e, t = now.t;
    int pos = t;
    if (S == kRowsOut) {
      if (a.positions) pos = a.positions[now.token];
    } else {
      if (p.parent) pos = node_depth(p.parent + static_cast<size_t>(e) * a.T, a.T, t, p.v.err);
      pos += p.plan[e * kPlanInts + 2];
    }
    float cs[8], sn[8];
    {
      float c[PPL], s[PPL];
#pragma unroll
      for (int i = 0; i < PPL; ++i) {
        const uint64_t x = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns[i];
        sincospif(static_cast<float>(static_cast<int32_t>(x >> 32)) * 0x1p-31f, &s[i], &c[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // of pairs 8 l .. 8 l + 7, or of the four of each chunk
        const int pair = a.r.half ? 8 * l + i : 4 * (i < 4 ? c0 : c1) + (i & 3);
        cs[i] = __shfl_sync(0xffffffffu, c[i % PPL], pair / PPL) * a.r.factor;
        sn[i] = __shfl_sync(0xffffffffu, s[i % PPL], pair / PPL) * a.r.factor;
      }
    }
    // where this token's keys and values go
    size_t slot = 0;
    int page = 0, seq = 0, at = 0;
    if (S != kRowsOut) {
      seq = p.seqs[e];
      at = p.plan[e * kPlanInts + 1] + t;
      page = p.v.table[static_cast<size_t>(seq) * p.v.width + (at >> p.v.shift)];
      if (page < 0 || page >= p.v.pages) {
        atomicOr(p.v.err, kErrBadState);
        page = -1;
      }
      slot = ((static_cast<size_t>(max(page, 0)) * p.v.heads) << p.v.shift) + (at & (p.v.page - 1));
    }

    for (int i = now.i; i < now.last;) {
      const int kind = i < nq ? 0 : i < nk ? 1 : 2;
      const int end = min(now.last, kind == 0 ? nq : kind == 1 ? nk : rounds);
      int h = (i - (kind == 0 ? 0 : kind == 1 ? nq : nk)) * HEADS + g;
      const int heads = S != kRowsOut && kind && page < 0 ? 0 : a.heads[kind];
      const float* norm = kind < 2 ? a.norm[kind] : nullptr;
      float4 w[4];
      if (norm) {
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] = reinterpret_cast<const float4*>(norm)[(x < 2 ? c0 : c1) * 2 + (x & 1)];
      }
      // pages: of tokens of d channels in a head's page; rows: of a head's T tokens; queries: of a token's heads
      const bool paged = S != kRowsOut && kind;
      uint4* out = static_cast<uint4*>(paged ? static_cast<void*>(kind == 2 ? p.v.V : p.v.K) : a.out[kind]);
      const size_t first = paged ? slot
                           : S == kRowsOut ? static_cast<size_t>(e) * a.heads[kind] * a.T + t
                                           : static_cast<size_t>(now.token) * a.heads[kind];
      const size_t apart = paged ? p.v.page : S == kRowsOut ? a.T : 1;
      for (; i < end; ++i, h += HEADS, st = st + 1 < kStages ? st + 1 : 0) {
        copy_async_wait<kStages - 2>();
        uint4 raw[2] = {ring[st * 64], ring[st * 64 + 32]};
        fetch(st ? st - 1 : kStages - 1);  // into the slot of the round before
        if (h < heads) {  // (whole heads: the lanes of one go the same way)
          const size_t to = first + h * apart;
          float f[16];
          if (kind < 2 || S == kPagesF8) {
            bf16x8_to_f32(raw[0], f);
            bf16x8_to_f32(raw[1], f + 8);
          }
          if (norm) {
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < 16; ++x) sum = fmaf(f[x], f[x], sum);
#pragma unroll
            for (int off = LPR / 2; off; off >>= 1) sum += __shfl_xor_sync(gmask, sum, off);
            const float inv = rsqrtf(fmaf(sum, 1.f / D, a.eps));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              f[4 * x] *= inv * w[x].x;
              f[4 * x + 1] *= inv * w[x].y;
              f[4 * x + 2] *= inv * w[x].z;
              f[4 * x + 3] *= inv * w[x].w;
            }
          }
          if (kind < 2) {
            if (a.r.half) {
              if (turn0) {
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  const float y = f[x], z = f[8 + x];
                  f[x] = y * cs[x] - z * sn[x];
                  f[8 + x] = y * sn[x] + z * cs[x];
                }
              }
            } else {
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                if (!(x < 4 ? turn0 : turn1)) continue;
                const float y = f[2 * x], z = f[2 * x + 1];
                f[2 * x] = y * cs[x] - z * sn[x];
                f[2 * x + 1] = y * sn[x] + z * cs[x];
              }
            }
            if (paged && l == 0) {
              p.v.pos[to] = pos;
              p.v.score[(static_cast<size_t>(seq) * p.v.heads + h) * p.v.cap + at] = 0.f;
            }
          }
          if (S == kPagesF8 && kind) {
            // a NaN or an infinity has no code: the vector becomes NaN by its scale
            bool wild = false;
#pragma unroll
            for (int x = 0; x < 16; ++x) wild |= !(fabsf(f[x]) < INFINITY);
            wild = __ballot_sync(gmask, wild) & gmask;
            if (wild) {
#pragma unroll
              for (int x = 0; x < 16; ++x) f[x] = 0.f;
            }
            uint32_t pairs[8];
            float sc = quantize_e4m3<16>(f, gmask, LPR, pairs, kTinyVector);
            if (wild) sc = __int_as_float(0x7fc00000);
            uint2* dst = reinterpret_cast<uint2*>(out) + to * (D / 8);
            dst[c0] = make_uint2(pairs[0] | (pairs[1] << 16), pairs[2] | (pairs[3] << 16));
            dst[c1] = make_uint2(pairs[4] | (pairs[5] << 16), pairs[6] | (pairs[7] << 16));
            if (l == 0) (kind == 2 ? p.v.vscale : p.v.kscale)[to] = sc;
          } else {
            if (kind < 2) {
#pragma unroll
              for (int x = 0; x < 2; ++x)
                raw[x] = make_uint4(pack_bf16x2(f[8 * x], f[8 * x + 1]), pack_bf16x2(f[8 * x + 2], f[8 * x + 3]),
                                    pack_bf16x2(f[8 * x + 4], f[8 * x + 5]), pack_bf16x2(f[8 * x + 6], f[8 * x + 7]));
            }
            uint4* dst = out + to * (D / 8);
            dst[c0] = raw[0];
            dst[c1] = raw[1];
          }
        }
        __syncwarp();
      }
    }
  }
  copy_async_wait<0>();
}

template <Sink S>
cudaError_t rotate(const RotateArgs& a, const Pages& p, cudaStream_t stream) {
  const int64_t tokens = static_cast<int64_t>(a.n) * a.T;
  const int heads = 512 / a.d;
  int rounds = 0;
  for (int i = 0; i < 3; ++i) rounds += (a.heads[i] + heads - 1) / heads;
  if (tokens == 0 || rounds == 0) return cudaSuccess;
  // A token's rounds are dealt to several warps where there are fewer tokens than warps.
  const int64_t warps = static_cast<int64_t>(num_sms()) * kBlocks * (kThreads / 32);
  int parts = 1;
  while (parts < rounds && tokens * (parts + 1) <= warps) ++parts;
  const int64_t blocks = std::min(warps, tokens * parts + kThreads / 32 - 1) / (kThreads / 32);
  auto kern = a.d == 128 ? rotate_kernel<128, S> : rotate_kernel<64, S>;
  return launch_after(kern, dim3(static_cast<unsigned>(blocks)), kThreads, 0, stream, a, p, parts);
}

}  // namespace

cudaError_t rotate_qkv(const RotateArgs& a, cudaStream_t stream) { return rotate<kRowsOut>(a, Pages{}, stream); }

cudaError_t pool_append(const PoolView& v, const RotateArgs& a, const int32_t* seqs, const int32_t* lens,
                        const int32_t* parent, int32_t* fresh, int32_t* plan, cudaStream_t stream) {
  if (a.n == 0) return cudaSuccess;
  // (rows of queries that belong to no written token stay as they were)
  const int mark = kRefused | (a.heads[0] ? kRefusedQueries : 0);
  cudaError_t e = pool_write_plan(v, a.n, seqs, a.T, lens, parent != nullptr, mark, fresh, plan, stream);
  if (e != cudaSuccess || a.T == 0) return e;
  const Pages p{v, seqs, plan, parent};
  return v.kscale ? rotate<kPagesF8>(a, p, stream) : rotate<kPagesBf16>(a, p, stream);
}

}  // namespace h2o
