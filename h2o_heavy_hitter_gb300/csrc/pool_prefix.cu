// Attention over a prefix that many query rows share: the queries of all
// sequences of a batch are the rows of one matrix per key head. (The few-rows
// case, the own tokens and the joining of pieces are in pool_attend.cu.)
//
// pool_prefix_kernel: S = Q K^T and O += P V (tcgen05, accumulators in TMEM), a
//   thread per query row. Units are blocks of two tiles of 128 rows; a persistent
//   CTA per SM takes an equal contiguous share of the units' key tiles. With one
//   row tile the four warps of half t take keys 64 t .. 64 t + 63 of every tile and
//   an accumulator of their own, so that two short softmax chains run side by side
//   and no maximum is exchanged; with two, the halves take a row tile each and
//   share the key and value tiles. S is double-buffered: the product of the next
//   tile runs under the softmax of this one. P is two bf16 terms (pool_attend.cu), side
//   by side in the columns that S held. Bound by HBM up to some 128 rows,
//   beyond by the exponentials and the products of 256 rows a tile: 512 rows a
//   head, 8 heads, 32768 keys take 97 us with the joining (706 TFLOP/s, the products
//   with the second terms not counted). At 1024 keys a CTA has two tiles, and 17 us are
//   its start and the read-out.
// pool_prefix_score_kernel: the prefix's scores once the pieces are there: S^T = K
//   Q^T again, a thread per key, p = 2^(s - lse) summed over all rows in order. It
//   reads K once more (2 d bytes a key and head); keeping the logits of more than
//   32 rows would move 8 bytes a key and row. For up to 256 rows it joins the rows'
//   sums itself and runs beside the finish kernel (256 sequences: 290 -> 286 us in all).
#include "device_state.h"
#include "pool_tiles.cuh"

namespace h2o {
namespace {

// Whole 32-byte sectors: the rows of a warp's threads lie 4 D bytes apart, and with
// 16-byte stores the read-out of a unit took 4700 clocks.
__device__ __forceinline__ void store_32b(float* dst, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// ------------------------------------------------------------------ attention
// Warps: 0 tiles of keys or codes by TMA, 1 MMA and TMEM, 2 queries, 3 tiles of
// values, 4..7 half or row tile 0, 8..11: 1 (one per TMEM lane quadrant), 12..15
// E4M3 codes to bf16 tiles.
constexpr int kWarpMMA = 1, kWarpQ = 2, kWarpV = 3, kWarpSoftmax = 4, kWarpCodes = 12;
constexpr int kCodeThreads = 128;

template <int RK, int RV, int S>
struct Bars {
  RingBars<RK> keys;
  RingBars<RV> values;
  RingBars<S> codes;
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_ready[2], pv_done[2];  // by S buffer
  uint64_t o_last[2], o_free[2];               // one phase per unit
  uint64_t drained;
  uint32_t tmem;
};

template <int D, bool F8>
struct Cfg {
  static constexpr int THREADS = 32 * kWarpCodes + (F8 ? kCodeThreads : 0);
  static constexpr int TILE = TILE_KEYS * D * 2;
  static constexpr int KTILE = F8 ? TILE_KEYS * D : TILE;  // keys are used as they are stored
  static constexpr int RK = (F8 ? 3 : 2) * (128 / D), RV = (F8 ? 2 : 3) * (128 / D);
  static constexpr int S = F8 ? 2 * (128 / D) : 1;  // slots of value codes
  static constexpr int CODES = F8 ? S * TILE_KEYS * D : 0;
  static constexpr uint32_t O_COL = 256;  // S buffers at columns 0 and 128, O of half t at 256 + 128 t
  static constexpr int SCALES = F8 ? (RK + S + kScaleTiles) * TILE_KEYS * 4 : 0;
  static constexpr size_t SMEM = static_cast<size_t>(2 + RV) * TILE + RK * KTILE + CODES + SCALES +
                                 sizeof(Bars<RK, RV, S>) + 1024;
};

// A walk along one CTA's share of the units.
struct Walk {
  const AttendParams& p;
  int len, tiles, cta;
  int64_t at, end;
  bool two;
  int h, b, kt0, kt1, piece;

  __device__ Walk(const AttendParams& p, int len, int cta) : p(p), len(len), cta(cta) {
    tiles = key_tiles(len);
    const int64_t total = static_cast<int64_t>(p.s.heads) * p.s.blocks * tiles;
    at = share_begin(total, p.s.grid, cta);
    end = share_begin(total, p.s.grid, cta + 1);
  }
  __device__ int rows(int t) const {  // valid rows of the unit's row tile t
    return min(p.s.per_tile, p.s.n - (2 * b + (two ? t : 0)) * p.s.per_tile) * p.s.group;
  }
  __device__ bool next() {
    if (at >= end) return false;
    const int u = static_cast<int>(at / tiles);
    kt0 = static_cast<int>(at - static_cast<int64_t>(u) * tiles);
    kt1 = static_cast<int>(min(static_cast<int64_t>(tiles), kt0 + (end - at)));
    h = u / p.s.blocks;
    b = u - h * p.s.blocks;
    two = 2 * b + 1 < p.s.nq;
    piece = u + cta;
    at += kt1 - kt0;
    return true;
  }
};

struct TileCursor {
  Walk w;
  int kt, kt1, seq, len, h;
  __device__ explicit TileCursor(const Walk& walk)
      : w(walk), kt(-1), kt1(0), seq(walk.p.a.prefix), len(walk.len) {}
  __device__ bool step() {
    if (++kt < kt1) return true;
    if (!w.next()) return false;
    kt = w.kt0;
    kt1 = w.kt1;
    h = w.h;
    return true;
  }
};

template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::THREADS, 1)
    pool_prefix_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tq2,
                       const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv,
                       const __grid_constant__ AttendParams p) {
  using C = Cfg<D, F8>;
  constexpr int RK = C::RK, RV = C::RV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + 2 * C::TILE;
  uint8_t* sV = sK + RK * C::KTILE;
  uint8_t* codes = sV + RV * C::TILE;
  float* kscales = reinterpret_cast<float*>(codes + C::CODES);  // [RK][128]
  float* cscales = kscales + RK * TILE_KEYS;                    // [S][128], of value codes
  float* vscales = cscales + C::S * TILE_KEYS;                  // [kScaleTiles][128]
  auto* bars = reinterpret_cast<Bars<RK, RV, C::S>*>(reinterpret_cast<uint8_t*>(kscales) + C::SCALES);
  const PoolView& v = p.a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  grid_dependency_wait();
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
    for (int i = 0; i < RK; ++i) {
      mbar_init(&bars->keys.full[i], 1);
      mbar_init(&bars->keys.empty[i], F8 ? 1 + 8 : 1);  // the products, and the readers of the scales
    }
    for (int i = 0; i < RV; ++i) {
      mbar_init(&bars->values.full[i], F8 ? kCodeThreads / 32 : 1);
      mbar_init(&bars->values.empty[i], 1);
    }
    for (int i = 0; i < C::S; ++i) {
      mbar_init(&bars->codes.full[i], 1);
      mbar_init(&bars->codes.empty[i], kCodeThreads / 32);
    }
    mbar_init(&bars->drained, 1);
    fence_barrier_init();
  }
  if (warp == kWarpMMA) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
  }
  if (warp == kWarpQ && lane == 0) tma_prefetch_map(&tq);
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tk);
    tma_prefetch_map(&tv);
  }
  const int plen = max(0, checked_length(v, p.a.prefix, cta + threadIdx.x == 0));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  Walk w(p, plen, cta);
  if (threadIdx.x == 0) grid_release_dependents();  // the rows kernel, as SMs become free, does not wait first

  if (warp == 0) {
    if constexpr (F8)
      produce_codes<D, false>(v, &tk, v.kscale, sK, kscales, bars->keys, TileCursor(w));
    else
      produce_tma<D, false>(v, &tk, sK, bars->keys, TileCursor(w));
  } else if (warp == kWarpV) {
    if constexpr (F8)
      produce_codes<D, false>(v, &tv, v.vscale, codes, cscales, bars->codes, TileCursor(w));
    else
      produce_tma<D, false>(v, &tv, sV, bars->values, TileCursor(w));
  } else if (F8 && warp >= kWarpCodes) {
    convert_values<D, RV, C::S, kCodeThreads>(v, codes, cscales, bars->codes, sV, bars->values, vscales,
                                              TileCursor(w), threadIdx.x - 32 * kWarpCodes);
  } else if (warp == kWarpQ) {
    if (lane == 0) {
      uint32_t qn = 0;
      bool ok = true;
      while (ok && w.next()) {
        for (int t = 0; t < (w.two ? 2 : 1); ++t, ++qn) {
          const uint32_t qb = qn & 1;
          if (qn >= 2 && !pool_wait(&bars->q_empty[qb], ((qn >> 1) - 1) & 1, v.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars->q_full[qb], p.s.per_tile * p.s.group * D * 2);
          // boxes of 64 channels, or the two codes of every value
#pragma unroll
          for (int c = 0; c < (F8 ? 2 : D / 64); ++c)
            tma_load_4d(sQ + qb * C::TILE + c * (F8 ? C::KTILE : kBoxBytes), c == 1 && F8 ? &tq2 : &tq,
                        F8 ? 0 : c * 64, 0, w.h, (2 * w.b + t) * p.s.per_tile, &bars->q_full[qb]);
        }
      }
      drain_copies(bars->q_full, qn, v.err);
    }
  } else if (warp == kWarpMMA) {
    // ---------------------------------------------------------------- MMA issuer
    // S j is followed by the P V of S j - 1, so the softmax of one S overlaps the
    // product of the next; the S buffer of j is that of j - 2, whose P V is issued.
    {
      constexpr uint32_t idesc_qk = idesc_bf16(TILE_ROWS, TILE_KEYS, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16(TILE_ROWS, D, 0, 1);
      const uint64_t dq0 = F8 ? desc_codes<D>(sQ) : desc_kmajor<D>(sQ, 0);
      const uint64_t dk0 = F8 ? desc_codes<D>(sK) : desc_kmajor<D>(sK, 0);
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
        const uint32_t st = pv.g % RV, buf = pv.j & 1;
        if (!pool_warp_wait(&bars->p_ready[buf], (pv.j >> 1) & 1, v.err) ||
            !pool_warp_wait(&bars->values.full[st], (pv.g / RV) & 1, v.err))
          return false;
        if (pv.first && pv.e > 0) {
          for (int t = 0; t < 2; ++t)
            if ((!pv.two || t == pv.t) && !pool_warp_wait(&bars->o_free[t], (pv.e - 1) & 1, v.err))
              return false;
        }
        tc_fence_after();
        const uint64_t vb = dv0 + static_cast<uint64_t>(st * (C::TILE >> 4));
        const uint32_t s_tm = tmem + buf * 128;
        if (elect_one()) {
          // B = V tile, MN-major: 16 keys = two 8-row swizzle atoms (2048 bytes)
#pragma unroll
          for (int kk = 0; kk < TILE_KEYS / 16; ++kk) {
            const int half = kk >> 2;
            const uint32_t o = tmem + C::O_COL + (pv.two ? pv.t : half) * 128;
            const uint32_t a = s_tm + half * 64 + (kk & 3) * 8;
            const bool fresh = pv.first && (pv.two ? kk == 0 : (kk & 3) == 0);
            umma_ts(o, a, vb + kk * (2048 >> 4), idesc_pv, fresh ? 0u : 1u);
            umma_ts(o, a + 32, vb + kk * (2048 >> 4), idesc_pv, 1u);  // the second term
          }
          umma_commit(&bars->pv_done[buf]);
          if (pv.frees) umma_commit(&bars->values.empty[st]);
          if (pv.last)
            for (int t = 0; t < 2; ++t)
              if (!pv.two || t == pv.t) umma_commit(&bars->o_last[t]);
        }
        __syncwarp();
        return true;
      };
      while (ok && w.next()) {
        const int nt = w.two ? 2 : 1;
        for (int kt = w.kt0; ok && kt < w.kt1; ++kt, ++g) {
          const uint32_t st = g % RK;
          for (int t = 0; ok && t < nt; ++t, ++j) {
            const uint32_t qb = (qn + t) & 1;
            if ((kt == w.kt0 && !pool_warp_wait(&bars->q_full[qb], ((qn + t) >> 1) & 1, v.err)) ||
                (t == 0 && !pool_warp_wait(&bars->keys.full[st], (g / RK) & 1, v.err))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t kb = dk0 + static_cast<uint64_t>(st * (C::KTILE >> 4));
            const uint64_t qd = dq0 + static_cast<uint64_t>(qb * (C::TILE >> 4));
            const uint32_t d_tm = tmem + (j & 1) * 128;
            if (elect_one()) {
              if constexpr (F8) {
#pragma unroll
                for (int kk = 0; kk < 2 * (D / 32); ++kk)  // the queries' first codes, then their second
                  umma_ss_8bit(d_tm, qd + kk / (D / 32) * (C::KTILE >> 4) + kk % (D / 32) * 2,
                               kb + kk % (D / 32) * 2, idesc_e4m3(TILE_ROWS, TILE_KEYS), kk > 0);
              } else {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                  const uint64_t off = ((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4;
                  umma_ss(d_tm, qd + off, kb + off, idesc_qk, kk > 0);
                }
              }
              umma_commit(&bars->s_full[j & 1]);
              if (t == nt - 1) umma_commit(&bars->keys.empty[st]);
              if (kt == w.kt1 - 1) umma_commit(&bars->q_empty[qb]);
            }
            __syncwarp();
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
      drain_products(&bars->drained, v.err);
    }
  } else if (warp >= kWarpSoftmax && warp < kWarpCodes) {
    // ---------------------------------------------------------------- softmax
    const int t = (warp - kWarpSoftmax) >> 2, quad = warp & 3;
    const int r = quad * 32 + lane, tid = ((warp - kWarpSoftmax) & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t o_tm = tmem + lane_off + C::O_COL + t * 128;
    uint32_t j0 = 0, g = 0;
    int e = 0;
    bool ok = true;
    while (ok && w.next()) {
      const int rows = w.rows(t), step = w.two ? 2 : 1;
      const bool active = quad * 32 < rows;  // warp-uniform
      const int chunks = w.two ? 2 : 1, col0 = w.two ? 0 : 64 * t;
      // bf16: of all logits, in the exponent's product; E4M3: of the row's codes, in the key's scale
      // (their product stays in range where a key's times the sum of codes need not)
      float m = -INFINITY, l = 0.f, rscale = p.qscale;
      const float qscale = F8 ? 1.f : p.qscale;
      if (F8 && r < rows) {
        const int entry = (2 * w.b + (w.two ? t : 0)) * p.s.per_tile + r / p.s.group;
        rscale *= p.w.qfac[(static_cast<size_t>(entry) * p.s.heads + w.h) * p.s.group + r % p.s.group];
      }
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++g) {
        const uint32_t jj = j0 + (kt - w.kt0) * step, j = w.two ? jj + t : jj;
        const uint32_t s_tm = tmem + lane_off + (j & 1) * 128, st = g % RV;
        if (!pool_warp_wait(&bars->s_full[j & 1], (j >> 1) & 1, v.err)) {
          ok = false;
          break;
        }
        const int valid = w.len - kt * TILE_KEYS;  // may exceed 128
        // the value tile stays in its slot until these probabilities are used; the
        // keys' product is done, so their tile has arrived, and it stays until the arrival below
        if ((F8 && !pool_warp_wait(&bars->keys.full[g % RK], (g / RK) & 1, v.err)) ||
            ((F8 || valid < TILE_KEYS) &&
             !pool_warp_wait(&bars->values.full[st], (g / RV) & 1, v.err))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const ulonglong2* ks = reinterpret_cast<const ulonglong2*>(kscales + g % RK * TILE_KEYS);
        const uint64_t rs = f2_pack(rscale, rscale);
        const float4* vs = reinterpret_cast<const float4*>(vscales + g % kScaleTiles * TILE_KEYS);
        // 64 logits from column `first`, (bf16) unscaled by 1 / sqrt(d); those behind the end -inf
        auto load = [&](uint32_t (&s)[64], int first) {
          tmem_ld32(s_tm + first, s);
          tmem_ld32(s_tm + first + 32, s + 32);
          tmem_wait_ld();
          if (F8) {
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const ulonglong2 k4 = ks[first / 4 + x];
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int i = 4 * x + 2 * y;
                float a, b;
                f2_unpack(f2_mul(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])),
                                 f2_mul(y ? k4.y : k4.x, rs)),
                          a, b);
                s[i] = __float_as_uint(a);
                s[i + 1] = __float_as_uint(b);
              }
            }
          }
          if (first + 64 > valid) {
#pragma unroll
            for (int x = 0; x < 64; ++x)
              if (first + x >= valid) s[x] = __float_as_uint(-INFINITY);
          }
        };
        if (active) {
          uint32_t s[64];
          float mx = -INFINITY;
          for (int c = 0; c < chunks; ++c) {
            const int first = col0 + 64 * c;
            load(s, first);
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int x = 0; x < 64; x += 8)
#pragma unroll
              for (int y = 0; y < 4; ++y)
                m4[y] = fmax3(m4[y], __uint_as_float(s[x + y]), __uint_as_float(s[x + 4 + y]));
            mx = fmax3(fmax3(mx, m4[0], m4[1]), m4[2], m4[3]);
          }
          mx *= qscale;
          float alpha = 1.f;
          bool rescale = false;
          if (mx > m + 8.f) {
            rescale = kt > w.kt0 && l > 0.f;
            if (rescale) alpha = ex2(m - mx);
            m = mx;
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const uint64_t sc2 = f2_pack(qscale, qscale), nm2 = f2_pack(-ref, -ref), minus = f2_pack(-1.f, -1.f);
          uint64_t rs2[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
          for (int c = chunks - 1; c >= 0; --c) {  // the last chunk is still in registers
            const int first = col0 + 64 * c;
            if (c < chunks - 1) load(s, first);
#pragma unroll
            for (int cc = 0; cc < 8; ++cc) {
              uint32_t pk[4], pk2[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int y = cc * 4 + x;
                float p0, p1;
                f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * y]), __uint_as_float(s[2 * y + 1])), sc2, nm2),
                          p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                rs2[x & 1] = f2_add(rs2[x & 1], f2_pack(p0, p1));
                if (F8) {
                  const float2 v2 = reinterpret_cast<const float2*>(vs)[first / 2 + y];
                  p0 *= v2.x;
                  p1 *= v2.y;
                }
                const uint32_t b0 = split_bits<F8>(p0), b1 = split_bits<F8>(p1);
                pk[x] = __byte_perm(b0, b1, 0x7632);
                f2_unpack(f2_fma(f2_pack(split_first(b0), split_first(b1)), minus,
                                 f2_pack(__uint_as_float(b0), __uint_as_float(b1))),
                          p0, p1);
                pk2[x] = pack_bf16x2(p0, p1);
              }
              // P over the S columns it came from: 32 of first terms, 32 of second
              tmem_st4(s_tm + first + cc * 4, pk);
              tmem_st4(s_tm + first + 32 + cc * 4, pk2);
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
            if (!w.two && !pool_warp_wait(&bars->pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, v.err)) {
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
        if (!F8 && valid < TILE_KEYS) {  // values behind the end count as zero, whatever they are
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
        if (lane == 0) {
          mbar_arrive_n(&bars->p_ready[j & 1], w.two ? 2 : 1);
          if (F8) mbar_arrive(&bars->keys.empty[g % RK]);
        }
      }
      if (!ok) break;
      // ---- the piece: O out of TMEM, which the next unit may then use
      if (!pool_warp_wait(&bars->o_last[t], e & 1, v.err)) break;
      tc_fence_after();
      if (active) {
        const size_t rec = (static_cast<size_t>(w.piece) * 2 + t) * TILE_ROWS + r;
        float* po = p.w.po + rec * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_tm + c * 32, o);
          tmem_wait_ld();
          if (r < rows) {
#pragma unroll
            for (int x = 0; x < 4; ++x) store_32b(po + c * 32 + 8 * x, o + 8 * x);
          }
        }
        if (r < rows) p.w.pml[rec] = make_float2(m, l);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_free[t]);
      j0 += (w.kt1 - w.kt0) * step;
      ++e;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ scores of the prefix
template <int R>
struct ScoreBars {
  RingBars<R> keys;
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[4], s_free[4];  // S buffers 2 t + (0, 1) of half t
  uint64_t joined;                // a phase per head of the share
  uint64_t drained;
  uint32_t tmem;
  // -lse [0] and the scale of the codes [1] of rows, which all lanes read at once: of a head's
  // rows, by heads & 1 (score_joins), or of the 32 rows that a warp has at hand
  alignas(16) float rows[2][2][2 * TILE_ROWS];
  alignas(16) float some[2][8][32];
};

// Warps as above, 4..7 even key tiles, 8..11 odd ones.
template <int D, bool F8>
struct ScoreCfg {
  static constexpr int THREADS = 32 * kWarpCodes;
  static constexpr int TILE = TILE_KEYS * D * 2;
  static constexpr int KTILE = F8 ? TILE_KEYS * D : TILE;
  static constexpr int R = (F8 ? 8 : 4) * (128 / D);
  static constexpr int SCALES = F8 ? R * TILE_KEYS * 4 : 0;
  static constexpr size_t SMEM =
      static_cast<size_t>(2) * TILE + R * KTILE + SCALES + sizeof(ScoreBars<R>) + 1024;
};

// One CTA's share of the (head, key tile) list.
struct KeyCursor {
  int64_t it, end;
  int tiles, seq, len, h, kt;
  __device__ KeyCursor(const AttendParams& p, int len, int cta) : seq(p.a.prefix), len(len) {
    tiles = key_tiles(len);
    const int64_t total = static_cast<int64_t>(p.s.heads) * tiles;
    it = share_begin(total, p.s.grid, cta) - 1;
    end = share_begin(total, p.s.grid, cta + 1);
  }
  __device__ bool step() {
    if (++it >= end) return false;
    h = static_cast<int>(it / tiles);
    kt = static_cast<int>(it - static_cast<int64_t>(h) * tiles);
    return true;
  }
  // after step(): this is the head's last tile of the share
  __device__ bool last_of_head() const { return it + 1 >= end || kt + 1 == tiles; }
};

// E4M3: what the codes of an entry's query row are to be multiplied by.
__device__ __forceinline__ float row_factor(const AttendParams& p, int entry, int h, int g) {
  return p.w.qfac[(static_cast<size_t>(entry) * p.s.heads + h) * p.s.group + g];
}

// -lse (base 2) of row r of a head's row tile qt, -inf for one that is not counted.
__device__ __noinline__ float joined_row(const AttendParams& p, int qt, int r, int h, int len) {
  const int b = qt * p.s.per_tile + r / p.s.group, g = r % p.s.group;
  if (r >= p.s.per_tile * p.s.group || b >= p.s.n || p.w.seq[b] < 0) return -INFINITY;
  const int cum[3] = {p.w.cum[b], p.w.cum[b + 1], p.w.cum[p.s.n]};
  auto owners = [&](const int64_t (&at)[4], const int64_t (&total)[2], int (&c)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = total[i / 2] > 0 ? owner(at[i], total[i / 2], p.s.grid) : 0;
  };
  const Records x = place_records(p, b, h, len, cum, owners);
  const int all = x.prefix + x.own;
  float m = -INFINITY, l = 0.f;
  for (int i0 = 0; i0 < all; i0 += 8) {  // eight loads in flight
    float2 y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      y[i] = i0 + i < all ? record_ml(p, x, i0 + i, g) : make_float2(-INFINITY, 0.f);
    float top = m, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, y[i].x);
    const float ref = top == -INFINITY ? 0.f : top;  // (no logit but -inf: sums of zero, or a NaN)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += y[i].y * ex2(y[i].x - ref);
    l = l * ex2(m - ref) + sum;
    m = top;
  }
  return -(m + log2f(l));
}

// Fewer registers than THREADS threads could have (112 at most), so that three blocks of
// the finish kernel fit beside a CTA: grouped E4M3 heads 75.9 us a call (when P was one
// term), with 162 registers 84.4, with 80 and spills 77.9.
constexpr int kScoreBound = 576;

// The row tiles of a head stay in shared memory when there are at most two; more
// are fetched again for every key tile. A fill is one load of a row tile: fill f
// lies in buffer f & 1.
template <int D, bool F8>
__global__ void __launch_bounds__(kScoreBound, 1)
    pool_prefix_score_kernel(const __grid_constant__ CUtensorMap tq,
                             const __grid_constant__ CUtensorMap tq2,
                             const __grid_constant__ CUtensorMap tk,
                             const __grid_constant__ AttendParams p) {
  using C = ScoreCfg<D, F8>;
  constexpr int R = C::R;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint8_t* sQ = smem;
  uint8_t* ring = smem + 2 * C::TILE;
  float* scales = reinterpret_cast<float*>(ring + R * C::KTILE);  // [R][128]
  auto* bars = reinterpret_cast<ScoreBars<R>*>(reinterpret_cast<uint8_t*>(scales) + C::SCALES);
  const PoolView& v = p.a.v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    grid_acquire();  // the prefix's length, pages and queries; the softmax warps wait for the rest
    for (int i = 0; i < R; ++i) {
      mbar_init(&bars->keys.full[i], 1);
      mbar_init(&bars->keys.empty[i], F8 ? 1 + 4 : 1);  // the products, and the readers of the scales
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->q_empty[i], 1);
    }
    mbar_init(&bars->joined, 8);
    mbar_init(&bars->drained, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->s_free[i], 4);
    }
    fence_barrier_init();
  }
  if (warp == kWarpMMA) {
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
  const int len = max(0, checked_length(v, p.a.prefix, false));
  const int nq = p.s.nq, group = p.s.group;
  const bool stay = score_joins(p.s);
  KeyCursor k(p, len, blockIdx.x);

  if (warp == 0) {
    if constexpr (F8)
      produce_codes<D, false>(v, &tk, v.kscale, ring, scales, bars->keys, k);
    else
      produce_tma<D, false>(v, &tk, ring, bars->keys, k);
  } else if (warp == kWarpQ) {
    if (lane == 0) {
      uint32_t f = 0;
      int last = -1;
      bool ok = true;
      while (ok && k.step()) {
        if (stay && k.h == last) continue;
        last = k.h;
        for (int qt = 0; qt < nq; ++qt, ++f) {
          const uint32_t qb = f & 1;
          if (f >= 2 && !pool_wait(&bars->q_empty[qb], ((f >> 1) - 1) & 1, v.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars->q_full[qb], p.s.per_tile * group * D * 2);
#pragma unroll
          for (int c = 0; c < (F8 ? 2 : D / 64); ++c)
            tma_load_4d(sQ + qb * C::TILE + c * (F8 ? C::KTILE : kBoxBytes), c == 1 && F8 ? &tq2 : &tq,
                        F8 ? 0 : c * 64, 0, k.h, qt * p.s.per_tile, &bars->q_full[qb]);
        }
      }
      drain_copies(bars->q_full, f, v.err);
    }
  } else if (warp == kWarpMMA) {
    {
      const uint64_t dq0 = F8 ? desc_codes<D>(sQ) : desc_kmajor<D>(sQ, 0);
      const uint64_t dk0 = F8 ? desc_codes<D>(ring) : desc_kmajor<D>(ring, 0);
      uint32_t f0 = 0, cnt[2] = {0, 0};  // f0: fill of the head's (or tile's) row tile 0
      bool ok = true;
      int last = -1;
      for (uint32_t g = 0; ok && k.step(); ++g) {
        const bool fresh = !stay || k.h != last;  // row tiles newly filled
        if (fresh && last >= 0) f0 += nq;
        last = k.h;
        const bool done = !stay || k.last_of_head();  // the row tiles' last use
        const uint32_t st = g % R;
        const int t = g & 1;
        if (!pool_warp_wait(&bars->keys.full[st], (g / R) & 1, v.err)) break;
        for (int qt = 0; qt < nq; ++qt) {
          const uint32_t f = f0 + qt, qb = f & 1, buf = 2 * t + (cnt[t] & 1);
          if ((fresh && !pool_warp_wait(&bars->q_full[qb], (f >> 1) & 1, v.err)) ||
              (cnt[t] >= 2 && !pool_warp_wait(&bars->s_free[buf], ((cnt[t] >> 1) - 1) & 1, v.err))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int rows = min(p.s.per_tile, p.s.n - qt * p.s.per_tile) * group;
          const int cols = (rows + 15) / 16 * 16;
          const uint64_t kb = dk0 + static_cast<uint64_t>(st * (C::KTILE >> 4));
          const uint64_t qd = dq0 + static_cast<uint64_t>(qb * (C::TILE >> 4));
          const uint32_t d_tm = tmem + buf * 128;
          if (elect_one()) {
            if constexpr (F8) {
              const uint32_t idesc = idesc_e4m3(TILE_KEYS, cols);
#pragma unroll
              for (int kk = 0; kk < 2 * (D / 32); ++kk)
                umma_ss_8bit(d_tm, kb + kk % (D / 32) * 2,
                             qd + kk / (D / 32) * (C::KTILE >> 4) + kk % (D / 32) * 2, idesc, kk > 0);
            } else {
              const uint32_t idesc = idesc_bf16(TILE_KEYS, cols, 0, 0);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t off = ((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4;
                umma_ss(d_tm, kb + off, qd + off, idesc, kk > 0);
              }
            }
            umma_commit(&bars->s_full[buf]);
            if (done) umma_commit(&bars->q_empty[qb]);
            if (qt == nq - 1) umma_commit(&bars->keys.empty[st]);
          }
          __syncwarp();
          ++cnt[t];
        }
      }
      drain_products(&bars->drained, v.err);
    }
  } else if (warp >= kWarpSoftmax && warp < kWarpCodes) {
    const int t = (warp - kWarpSoftmax) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t cnt = 0;
    bool ok = true;
    grid_dependency_wait();     // the pieces, or the lse's, by the kernels before
    // the finish kernel, when it comes behind this one, reads them at once
    if (warp == kWarpSoftmax && lane == 0) grid_release_dependents();
    int last = -1;
    uint32_t heads = 0;        // of the share so far
    for (uint32_t g = 0; ok && k.step(); ++g) {
      if (stay && last != k.h) {  // half t joins the rows of row tile t, both use them
        // (two buffers: the one written was last read before the other's phase)
        if (t < nq) {
          const int entry = t * p.s.per_tile + r / group;
          const int at = t * TILE_ROWS + r;
          if (F8) bars->rows[1][heads & 1][at] = entry < p.s.n ? row_factor(p, entry, k.h, r % group) : 1.f;
          bars->rows[0][heads & 1][at] = joined_row(p, t, r, k.h, len);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->joined);
        if (!pool_warp_wait(&bars->joined, heads & 1, v.err)) break;
        ++heads;
        last = k.h;
      }
      if ((g & 1) != static_cast<uint32_t>(t)) continue;
      float acc = 0.f, ks = p.qscale;
      for (int qt = 0; qt < nq; ++qt, ++cnt) {
        const uint32_t buf = 2 * t + (cnt & 1);
        const int rows = min(p.s.per_tile, p.s.n - qt * p.s.per_tile) * group;
        if (!pool_warp_wait(&bars->s_full[buf], (cnt >> 1) & 1, v.err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (F8 && qt == 0) {  // the tile has arrived, and stays until the arrival here
          if (!pool_warp_wait(&bars->keys.full[g % R], (g / R) & 1, v.err)) {
            ok = false;
            break;
          }
          ks = p.qscale * scales[g % R * TILE_KEYS + r];
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->keys.empty[g % R]);
        }
        float part[4] = {0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < rows; c += 32) {
          const float* nl = bars->rows[0][(heads - 1) & 1] + qt * TILE_ROWS + c;
          const float* fac = bars->rows[1][(heads - 1) & 1] + qt * TILE_ROWS + c;
          if (!stay) {
            nl = bars->some[0][warp - kWarpSoftmax];
            fac = bars->some[1][warp - kWarpSoftmax];
            const int at = c + lane;
            const bool in = at < rows;
            const float mine =
                in ? p.w.nlse[(static_cast<size_t>(k.h) * nq + qt) * TILE_ROWS + at] : -INFINITY;
            const float mf =
                F8 && in ? row_factor(p, qt * p.s.per_tile + at / group, k.h, at % group) : 1.f;
            __syncwarp();
            bars->some[0][warp - kWarpSoftmax][lane] = mine;
            if (F8) bars->some[1][warp - kWarpSoftmax][lane] = mf;
            __syncwarp();
          }
          uint32_t s[32];
          tmem_ld32(tmem + lane_off + buf * 128 + c, s);
          tmem_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const float4 n4 = *reinterpret_cast<const float4*>(nl + x);
            const float4 f4 =
                F8 ? *reinterpret_cast<const float4*>(fac + x) : make_float4(1.f, 1.f, 1.f, 1.f);
            const float n[4] = {n4.x, n4.y, n4.z, n4.w}, f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              // rows that are not counted, and columns that are none, may hold anything
              const float e = ex2(fmaf(__uint_as_float(s[x + y]), F8 ? ks * f[y] : ks, n[y]));
              part[y] += n[y] == -INFINITY ? 0.f : e;
            }
          }
        }
        acc += (part[0] + part[1]) + (part[2] + part[3]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_free[buf]);
      }
      if (!ok) break;
      const int key = k.kt * TILE_KEYS + r;
      if (key < len) v.score[(static_cast<size_t>(p.a.prefix) * v.heads + k.h) * v.cap + key] += acc;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host side
template <int D, bool F8>
cudaError_t prefix_t(const AttendParams& p, cudaStream_t stream) {
  CUtensorMap tq, tq2;
  const CUtensorMap &tk = *p.a.kmap, &tv = *p.a.vmap;
  cudaError_t e = F8 ? query_code_map(&tq, p, 0, p.s.per_tile) : query_map(&tq, p.a, p.s.per_tile);
  if (e == cudaSuccess && F8) e = query_code_map(&tq2, p, 1, p.s.per_tile);
  if (!F8) tq2 = tq;
  if (e != cudaSuccess) return e;
  using C = Cfg<D, F8>;
  static int opted_in[kMaxDevices] = {};
  if ((e = raise_smem_limit(reinterpret_cast<const void*>(pool_prefix_kernel<D, F8>), C::SMEM,
                            opted_in)) != cudaSuccess)
    return e;
  return launch_after(pool_prefix_kernel<D, F8>, dim3(p.s.grid), C::THREADS, C::SMEM, stream, tq, tq2, tk,
                      tv, p);
}

template <int D, bool F8>
cudaError_t score_t(const AttendParams& p, cudaStream_t stream) {
  CUtensorMap tq, tq2;
  const CUtensorMap& tk = *p.a.kmap;
  cudaError_t e = F8 ? query_code_map(&tq, p, 0, p.s.per_tile) : query_map(&tq, p.a, p.s.per_tile);
  if (e == cudaSuccess && F8) e = query_code_map(&tq2, p, 1, p.s.per_tile);
  if (!F8) tq2 = tq;
  if (e != cudaSuccess) return e;
  using C = ScoreCfg<D, F8>;
  static int opted_in[kMaxDevices] = {};
  if ((e = raise_smem_limit(reinterpret_cast<const void*>(pool_prefix_score_kernel<D, F8>), C::SMEM,
                            opted_in)) != cudaSuccess)
    return e;
  return launch_after(pool_prefix_score_kernel<D, F8>, dim3(p.s.grid), C::THREADS, C::SMEM, stream,
                      tq, tq2, tk, p);
}

}  // namespace

cudaError_t pool_prefix(const AttendParams& p, cudaStream_t stream) {
  if (p.a.v.kscale) return p.s.d == 128 ? prefix_t<128, true>(p, stream) : prefix_t<64, true>(p, stream);
  return p.s.d == 128 ? prefix_t<128, false>(p, stream) : prefix_t<64, false>(p, stream);
}

cudaError_t pool_prefix_score(const AttendParams& p, cudaStream_t stream) {
  if (p.a.v.kscale) return p.s.d == 128 ? score_t<128, true>(p, stream) : score_t<64, true>(p, stream);
  return p.s.d == 128 ? score_t<128, false>(p, stream) : score_t<64, false>(p, stream);
}

}  // namespace h2o
