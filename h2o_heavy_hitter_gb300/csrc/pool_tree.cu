// Attention of a tree of drafted tokens over the paged cache: node t of a sequence
// attends to a shared prefix, to the sequence's tokens before its drafts, to the
// nodes of its branch and to itself. (The tiles' products are pool_prefix_kernel's,
// pool_prefix.cu; this file joins the pieces of units that several workers had.)
//
// Bound: a sequence's own keys and values are read once, 4 d bytes a token and head (2 d + 8 in
// E4M3), against 4 d flops a row, of which a head has nodes x group: HBM up to some 250 rows,
// tensor cores beyond. A prefix is read, and multiplied with whole row tiles, for every sequence:
// 64 sequences of 4 drafts, 8 heads of 128, over 32768 tokens take 985 us, where single tokens of
// the same sequences, whose rows share the tiles, take 66. Units are 256 rows (two row tiles
// share a tile of keys and values) or 128, where the CTA's two halves of softmax warps are
// workers of their own.
// A worker has an equal share of the tiles of all units; a unit that it has alone is
// written out from its accumulators, the at most two others of a worker become pieces,
// which the join kernel adds up by the records that the workers leave.
//
// Measured, all kernels of a call: four documents of 32768 tokens, 16 drafts, 32 heads of
// bf16 (2.1 GB) 322 us; 64 sequences of up to 2000 tokens and 32 drafts, 8 heads of E4M3
// with 4 query heads each 128 us; 256 rows a head over a prefix of 8197 keys 177 us; five
// drafts of one sequence 10 us.
#include <algorithm>

#include "device_state.h"
#include "pool_tree.cuh"

namespace h2o {
namespace {

constexpr int kJoinWarps = 8;

// Block (c, part): joins the unit that begins in worker c's share and goes on behind it, if there
// is one. A warp a row.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
    pool_tree_join_kernel(const __grid_constant__ AttendParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int worker = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const TreeCut u = p.w.cut[worker];
  if (u.pieces == 0) return;
  const int pieces = u.pieces, tiles = p.t.T * p.s.group > TILE_ROWS ? 2 : 1, q_heads = p.s.heads * p.s.group;
  const int rows = min(2 * p.s.per_tile, u.nodes - u.node) * p.s.group;
  for (int i = blockIdx.y * kJoinWarps + warp; i < rows; i += gridDim.y * kJoinWarps) {
    // a row tile holds per_tile nodes' rows, which may be fewer than 128
    const int tile = i / (p.s.per_tile * p.s.group), r = i - tile * p.s.per_tile * p.s.group;
    auto record = [&](int k) {
      return (static_cast<size_t>(2 * (worker + k) + (k == 0)) * tiles + tile) * TILE_ROWS + r;
    };
    float m = -INFINITY, l = 0.f;
    for (int k = lane; k < pieces; k += 32) {
      const float2 x = p.w.pml[record(k)];
      join(m, l, x.x, x.y);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m, off), l2 = __shfl_xor_sync(0xffffffffu, l, off);
      join(m, l, mo, l2);
    }
    const float lse = __shfl_sync(0xffffffffu, m + log2f(l), 0);
    float acc[D / 32] = {};
    for (int k0 = 0; k0 < pieces; k0 += 32) {
      const float wgt = k0 + lane < pieces ? ex2(p.w.pml[record(k0 + lane)].x - lse) : 0.f;
      const int count = min(32, pieces - k0);
#pragma unroll 4
      for (int k = 0; k < count; ++k) {
        const float wk = __shfl_sync(0xffffffffu, wgt, k);
        const float* o = p.w.po + record(k0 + k) * D + lane * (D / 32);
        float part[D / 32];
        if constexpr (D == 128) {
          const float4 y = *reinterpret_cast<const float4*>(o);
          part[0] = y.x, part[1] = y.y, part[2] = y.z, part[3] = y.w;
        } else {
          const float2 y = *reinterpret_cast<const float2*>(o);
          part[0] = y.x, part[1] = y.y;
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(wk, part[c], acc[c]);
      }
    }
    const size_t row =
        (static_cast<size_t>(u.b) * p.t.T + u.node + i / p.s.group) * q_heads + u.h * p.s.group + i % p.s.group;
    uint32_t* out = static_cast<uint32_t*>(p.a.out) + row * (D / 2) + lane * (D / 64);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) out[c] = pack_bf16x2(acc[2 * c], acc[2 * c + 1]);
    if (lane == 0 && p.a.lse) p.a.lse[row] = lse * 0.69314718055994531f;  // ln 2
  }
}

// s.n counts queries as a.n does: the queries' tensor map and codes are those of as many single tokens.
Shape tree_shape(const AttendArgs& a, const TreeArgs& t, int sms) {
  AttendParams p{};
  p.s.group = a.group;
  p.t = t;
  Shape s{};
  s.n = a.n;
  s.heads = a.v.heads;
  s.group = a.group;
  s.d = a.v.d;
  s.per_tile = TILE_ROWS / a.group;
  s.grid = tree_pairs(p) ? 2 * sms : sms;
  return s;
}

size_t scratch_layout(const Shape& s, const TreeArgs& t, bool codes, void* base, AttendScratch* out) {
  size_t at = 0;
  auto take = [&](size_t bytes) -> char* {
    if (!bytes) return nullptr;
    char* x = static_cast<char*>(base) + at;
    at += (bytes + 255) / 256 * 256;
    return x;
  };
  const size_t rows = static_cast<size_t>(s.grid) * 2 * (t.T * s.group > TILE_ROWS ? 2 : 1) * TILE_ROWS;
  const size_t queries = static_cast<size_t>(s.n) * s.heads * s.group;
  AttendScratch w{};
  w.cut = reinterpret_cast<TreeCut*>(take(s.grid * sizeof(TreeCut)));
  w.pml = reinterpret_cast<float2*>(take(rows * sizeof(float2)));
  w.po = reinterpret_cast<float*>(take(rows * s.d * sizeof(float)));
  w.q8 = reinterpret_cast<uint8_t*>(take(codes ? 2 * queries * s.d : 0));
  w.qfac = reinterpret_cast<float*>(take(codes ? queries * sizeof(float) : 0));
  if (out) *out = w;
  return at;
}

}  // namespace

size_t pool_tree_scratch(const AttendArgs& a, const TreeArgs& t) {
  return scratch_layout(tree_shape(a, t, num_sms()), t, a.v.kscale, nullptr, nullptr);
}

cudaError_t pool_tree(const AttendArgs& a, const TreeArgs& t, void* scratch, cudaStream_t stream) {
  if (t.n == 0 || t.T == 0) return cudaSuccess;
  AttendParams p{};
  p.a = a;
  p.t = t;
  p.s = tree_shape(a, t, num_sms());
  scratch_layout(p.s, t, a.v.kscale, scratch, &p.w);
  p.qscale = kLog2e / sqrtf(static_cast<float>(a.v.d));
  cudaError_t e;
  if (a.v.kscale && (e = pool_split_queries(p, stream)) != cudaSuccess) return e;
  // (a unit of one tile, and more no sequence of such a pool can have, is never in pieces)
  if ((e = pool_tree_rows(p, stream)) != cudaSuccess || (a.prefix < 0 && a.v.cap <= TILE_KEYS)) return e;
  const int rows = std::min(t.T * a.group, 2 * TILE_ROWS);
  return launch_after(a.v.d == 128 ? pool_tree_join_kernel<128> : pool_tree_join_kernel<64>,
                      dim3(p.s.grid, (rows + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0, stream, p);
}

}  // namespace h2o
