// Page management of the paged cache: writing tokens into sequences, forking,
// copying, freeing and compacting them.
//
// A page is free when no sequence holds it (ref 0); fresh pages are always the
// free ones of lowest index, given to the entries of a call's list in order, so
// a call's result depends on nothing but the pool's state. Every operation
// that needs pages runs a plan first: one block per layer, one thread per list
// entry, which checks the entries, counts what each needs, ranks the needs with
// a block scan, finds that many free pages in one pass over ref, and rewrites
// the tables. A second kernel then moves the tokens with the whole GPU. The
// passes over ref read four bytes a page and stop at the last page needed.
#include <algorithm>

#include "common.cuh"
#include "device_state.h"
#include "pool.h"
#include "scan.cuh"

namespace h2o {
namespace {

constexpr int kPlanThreads = 1024;
static_assert(kPlanThreads >= kPoolMaxList, "one thread per list entry");

__device__ __forceinline__ int pages_of(const PoolView& v, int tokens) {
  return (tokens + v.page - 1) >> v.shift;
}

// The view of one layer.
__device__ __forceinline__ PoolView at_layer(PoolView v, int layer) {
  const size_t slots = static_cast<size_t>(v.pages) * v.heads * v.page * layer;
  v.K += slots * v.row_bytes;
  v.V += slots * v.row_bytes;
  if (v.kscale) {
    v.kscale += slots;
    v.vscale += slots;
  }
  v.pos += slots;
  v.score += static_cast<size_t>(v.seqs) * v.heads * v.cap * layer;
  v.table += static_cast<size_t>(v.seqs) * v.width * layer;
  v.meta += static_cast<size_t>(v.seqs) * 2 * layer;
  v.ref += static_cast<size_t>(v.pages) * layer;
  return v;
}

// First slot (of heads * page per page) of a page's head.
__device__ __forceinline__ size_t slot_base(const PoolView& v, int page, int head) {
  return (static_cast<size_t>(page) * v.heads + head) << v.shift;
}

// A list entry: its sequence, or -1 when there is nothing to do. An index
// outside the pool, or one that an earlier entry names, is reported and skipped.
// Blockwide: s_list holds the list.
__device__ __forceinline__ int list_entry(const PoolView& v, const int32_t* list, int n,
                                          int* s_list) {
  const int i = threadIdx.x;
  int seq = i < n ? list[i] : -1;
  s_list[i] = seq;
  __syncthreads();
  if (seq == -1) return -1;
  bool bad = seq < 0 || seq >= v.seqs;
  for (int j = 0; j < i; ++j) bad |= s_list[j] == seq;
  if (bad) {
    atomicOr(v.err, kErrBadList);
    seq = -1;
  }
  return seq;
}

// A sequence's length; a state that no call leaves is reported and reads as refused (-1).
__device__ __forceinline__ int seq_length(const PoolView& v, int seq) {
  const int len = v.meta[2 * seq];
  if (len < 0 || len > v.cap) {
    atomicOr(v.err, kErrBadState);
    return -1;
  }
  return len;
}

// A page of a sequence, or -1 (reported) when the table holds none of the pool's.
__device__ __forceinline__ int held_page(const PoolView& v, int seq, int j) {
  const int p = v.table[static_cast<size_t>(seq) * v.width + j];
  if (p < 0 || p >= v.pages) {
    atomicOr(v.err, kErrBadState);
    return -1;
  }
  return p;
}

__device__ __forceinline__ void drop_page(const PoolView& v, int p) {
  if (atomicSub(&v.ref[p], 1) <= 0) {  // held by nobody: no call leaves that
    atomicAdd(&v.ref[p], 1);
    atomicOr(v.err, kErrBadState);
  }
}

// Finds the `total` free pages of lowest index, in order, into fresh[]; returns how many there are.
// Blockwide.
__device__ int find_free(const PoolView& v, int total, int32_t* fresh, int* wsum) {
  int found = 0;
  for (int base = 0; base < v.pages && found < total; base += 4 * kPlanThreads) {
    const int p = base + 4 * threadIdx.x;
    int r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = p + e < v.pages ? v.ref[p + e] : 1;
    const int mine = (r[0] == 0) + (r[1] == 0) + (r[2] == 0) + (r[3] == 0);
    int sum;
    int at = found + block_exclusive_scan(mine, wsum, &sum);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (r[e] == 0 && at < total) fresh[at++] = p + e;
    found += sum;
  }
  __syncthreads();  // fresh[] is visible to the block
  return min(found, total);
}

// Gives every entry its run of fresh pages: returns the run's first index, or
// -1 when the entry is refused because the free pages run out at it or before.
// Blockwide; need = 0 for entries without work.
__device__ int take_pages(const PoolView& v, int need, int32_t* fresh, int* wsum) {
  int total;
  const int first = block_exclusive_scan(need, wsum, &total);
  const int found = total ? find_free(v, total, fresh, wsum) : 0;
  return first + need <= found ? first : -1;
}

// How a block's warps go over the pages of n entries: a warp per entry, or several
// when there are fewer entries than warps.
struct Spread {
  int first, step;  // entries
  int lane, lanes;  // threads of an entry
  __device__ explicit Spread(int n) {
    constexpr int warps = kPlanThreads / 32;
    int per = 1;
    while (per < warps && n * per * 2 <= warps) per *= 2;
    lanes = 32 * per;
    first = threadIdx.x / lanes;
    step = warps / per;
    lane = threadIdx.x % lanes;
  }
};

// ------------------------------------------------------------------ fork, copy
constexpr int kSlab = 1024;  // slots of a sequence that the copy takes in one go, at least

// plan of an entry: {served, length, slabs (of kSlab) of the longest served entry, -}
__global__ void __launch_bounds__(kPlanThreads, 1)
    fork_plan_kernel(PoolView v0, int n, const int32_t* __restrict__ src,
                     const int32_t* __restrict__ dst, bool share, int32_t* fresh_all,
                     int fresh_stride, int32_t* plan_all) {
  __shared__ int s_list[kPlanThreads], s_src[kPlanThreads], s_len[kPlanThreads],
      s_first[kPlanThreads];
  __shared__ int wsum[33], longest;
  const PoolView v = at_layer(v0, blockIdx.x);
  int32_t* fresh = fresh_all + static_cast<size_t>(blockIdx.x) * fresh_stride;
  int32_t* plan = plan_all + static_cast<size_t>(blockIdx.x) * n * kPlanInts;
  const int i = threadIdx.x;
  if (i == 0) longest = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  int to = list_entry(v, dst, n, s_list);
  const int from = i < n ? src[i] : -1;
  int len = 0, next = 0;
  if (from == -1) to = -1;
  if (to >= 0) {
    // a source that is also a destination of this call is empty: both are read before any write
    if (from < 0 || from >= v.seqs || v.meta[2 * to] != 0) {
      atomicOr(v.err, kErrBadList);
      to = -1;
    } else if ((len = seq_length(v, from)) < 0) {
      to = -1;
    } else {
      next = v.meta[2 * from + 1];
    }
  }
  const int rest = len & (v.page - 1);
  const int need = to < 0 ? 0 : (share ? rest > 0 : pages_of(v, len));
  int first = take_pages(v, need, fresh, wsum);
  if (to >= 0 && first < 0) {
    atomicOr(v.err, kErrNoPages);
    to = -1;
  }
  s_list[i] = to;
  s_src[i] = from;
  s_len[i] = len;
  s_first[i] = first;
  if (to >= 0) atomicMax(&longest, len);
  __syncthreads();  // every length has been read
  if (i < n) {
    plan[i * kPlanInts] = to >= 0;
    plan[i * kPlanInts + 1] = len;
    plan[i * kPlanInts + 2] = (longest + kSlab - 1) / kSlab;
  }
  if (to >= 0) {
    v.meta[2 * to] = len;
    v.meta[2 * to + 1] = next;
  }
  const Spread w(n);
  for (int e = w.first; e < n; e += w.step) {
    const int b = s_list[e];
    if (b < 0) continue;
    const int whole = share ? s_len[e] >> v.shift : 0, np = pages_of(v, s_len[e]);
#pragma unroll 4
    for (int j = w.lane; j < np; j += w.lanes) {
      int p;
      if (j < whole) {
        p = held_page(v, s_src[e], j);
        if (p >= 0) atomicAdd(&v.ref[p], 1);
      } else {
        p = fresh[s_first[e] + j - whole];
        v.ref[p] = 1;
      }
      v.table[static_cast<size_t>(b) * v.width + j] = p;
    }
  }
}

// Copies `n` 16-byte chunks with LANES threads, four loads in flight per thread.
template <int LANES>
__device__ __forceinline__ void copy_chunks(uint8_t* dst, const uint8_t* src, int n, int lane) {
  int c = lane;
  for (; c + 3 * LANES < n; c += 4 * LANES) {
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = reinterpret_cast<const uint4*>(src)[c + LANES * u];
#pragma unroll
    for (int u = 0; u < 4; ++u) reinterpret_cast<uint4*>(dst)[c + LANES * u] = x[u];
  }
  for (; c < n; c += LANES) reinterpret_cast<uint4*>(dst)[c] = reinterpret_cast<const uint4*>(src)[c];
}

// n four-byte values, 16-byte aligned at both ends.
template <int LANES, typename T>
__device__ __forceinline__ void copy_values(T* dst, const T* src, int n, int lane) {
  copy_chunks<LANES>(reinterpret_cast<uint8_t*>(dst), reinterpret_cast<const uint8_t*>(src), n / 4, lane);
  const int rest = (n & ~3) + lane;
  if (rest < n) dst[rest] = src[rest];
}

// Copies the first `live` slots of a page's head.
template <int LANES>
__device__ __forceinline__ void copy_slots(const PoolView& v, int to, int from, int head, int live,
                                           int lane) {
  const size_t a = slot_base(v, from, head), b = slot_base(v, to, head);
  const int chunks = live * (v.row_bytes / 16);
  copy_chunks<LANES>(v.K + b * v.row_bytes, v.K + a * v.row_bytes, chunks, lane);
  copy_chunks<LANES>(v.V + b * v.row_bytes, v.V + a * v.row_bytes, chunks, lane);
  copy_values<LANES>(v.pos + b, v.pos + a, live, lane);
  if (v.kscale) {
    copy_values<LANES>(v.kscale + b, v.kscale + a, live, lane);
    copy_values<LANES>(v.vscale + b, v.vscale + a, live, lane);
  }
}

// LANES threads copy the slots [lo, hi) of an entry's head: their scores, and the tokens
// of their pages that were not shared. A head's slots of a page are contiguous, so a
// partial page is one run of bytes per head.
template <int LANES>
__device__ __forceinline__ void copy_slab(const PoolView& v, int from, int to, int head, int len, int lo,
                                          int hi, bool share, int lane) {
  copy_values<LANES>(v.score + (static_cast<size_t>(to) * v.heads + head) * v.cap + lo,
                     v.score + (static_cast<size_t>(from) * v.heads + head) * v.cap + lo, hi - lo, lane);
  const int first = share ? max(lo >> v.shift, len >> v.shift) : lo >> v.shift;
  for (int j = first; j << v.shift < hi; ++j) {
    const int a = held_page(v, from, j), b = held_page(v, to, j);
    if (a >= 0 && b >= 0) copy_slots<LANES>(v, b, a, head, min(v.page, len - (j << v.shift)), lane);
  }
}

// A warp per slab where the slabs that there are fill the GPU, else a block: 32 heads x 4
// entries of some 50 tokens take 7.6 us by blocks, 19.4 us by warps; 128 heads x 32768
// tokens (4096 slabs of kSlab) 33 us by blocks of 256 slots, 16 us by warps. The lengths
// decide, not what the sequences could hold.
constexpr int kManySlabs = 4096;

// LANES threads per unit (entry, head) and slab of `slab` slots: 32 where the units alone
// are many, else 256, one block or eight warps to the slab. Bound by HBM's writes and by a
// warp's loads behind one another: 56 forks of 8 prompts of 200 tokens, 48 layers of
// 56 heads, 1.1 GB in 207 us, each source read from HBM once. (Stores that leave L2 first
// made that 250 us; a loop over slabs of one size, with its registers, 225 us.)
template <int LANES>
__global__ void __launch_bounds__(256)
    fork_copy_kernel(PoolView v0, int n, const int32_t* __restrict__ src,
                     const int32_t* __restrict__ dst, bool share, int slab,
                     const int32_t* plan_all) {
  const PoolView v = at_layer(v0, blockIdx.z);
  const int32_t* plan = plan_all + static_cast<size_t>(blockIdx.z) * n * kPlanInts;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = LANES == 32 ? blockIdx.x * 8 + warp : blockIdx.x;
  const int e = unit / v.heads, head = unit % v.heads;
  grid_dependency_wait();
  grid_launch_dependents();
  if (e >= n || !plan[e * kPlanInts]) return;
  const int len = plan[e * kPlanInts + 1], lo = blockIdx.y * slab;
  if (lo >= len) return;
  const int from = src[e], to = dst[e];
  if (LANES == 32) {
    copy_slab<32>(v, from, to, head, len, lo, min(len, lo + slab), share, lane);
  } else if (static_cast<int64_t>(gridDim.x) * gridDim.z * plan[2] >= kManySlabs) {
    const int part = lo + warp * (slab / 8);  // whole pages
    if (part < len) copy_slab<32>(v, from, to, head, len, part, min(len, part + slab / 8), share, lane);
  } else {
    copy_slab<256>(v, from, to, head, len, lo, min(len, lo + slab), share, threadIdx.x);
  }
}

// ------------------------------------------------------------------ free
__global__ void __launch_bounds__(kPlanThreads)
    free_kernel(PoolView v0, int n, const int32_t* __restrict__ seqs) {
  __shared__ int s_list[kPlanThreads], s_len[kPlanThreads];
  const PoolView v = at_layer(v0, blockIdx.x);
  grid_dependency_wait();
  grid_launch_dependents();
  int seq = list_entry(v, seqs, n, s_list), len = 0;
  if (seq >= 0 && (len = seq_length(v, seq)) < 0) seq = -1;
  __syncthreads();  // every thread has compared the list
  s_list[threadIdx.x] = seq;
  s_len[threadIdx.x] = len;
  if (seq >= 0) *reinterpret_cast<int2*>(v.meta + 2 * seq) = make_int2(0, 0);
  __syncthreads();
  const Spread w(n);
  for (int e = w.first; e < n; e += w.step) {
    const int s = s_list[e];
    if (s < 0) continue;
    const int np = pages_of(v, s_len[e]);
#pragma unroll 4
    for (int j = w.lane; j < np; j += w.lanes) {
      const int p = held_page(v, s, j);
      if (p >= 0) drop_page(v, p);
      v.table[static_cast<size_t>(s) * v.width + j] = -1;
    }
  }
}

// ------------------------------------------------------------------ write
// plan of an entry: {tokens to write (0: none), first slot, first position, -}
__global__ void __launch_bounds__(kPlanThreads)
    write_plan_kernel(PoolView v, int n, const int32_t* __restrict__ seqs, int T,
                      const int32_t* __restrict__ lens, int32_t* fresh, int32_t* plan) {
  __shared__ int s_list[kPlanThreads], s_len[kPlanThreads], s_new[kPlanThreads],
      s_first[kPlanThreads];
  __shared__ int wsum[33];
  const int i = threadIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();
  int seq = list_entry(v, seqs, n, s_list);
  __syncthreads();
  int len = 0, next = 0, t = 0;
  if (seq >= 0) {
    t = lens ? lens[i] : T;
    if (t < 0 || t > T) {
      atomicOr(v.err, kErrBadLength);
      t = t < 0 ? 0 : T;
    }
    len = seq_length(v, seq);
    if (len < 0) {
      seq = -1;
    } else if (len + t > v.cap) {
      atomicOr(v.err, kErrNoPages);
      seq = -1;
    } else {
      next = v.meta[2 * seq + 1];
      // a partial last page belongs to its sequence alone
      if (t > 0 && (len & (v.page - 1))) {
        const int p = held_page(v, seq, len >> v.shift);
        if (p < 0 || v.ref[p] != 1) {
          atomicOr(v.err, kErrBadState);
          seq = -1;
        }
      }
    }
  }
  const int have = pages_of(v, max(len, 0));
  const int need = seq < 0 ? 0 : pages_of(v, len + t) - have;
  const int first = take_pages(v, need, fresh, wsum);
  if (seq >= 0 && first < 0) {
    atomicOr(v.err, kErrNoPages);
    seq = -1;
  }
  s_list[i] = seq;
  s_len[i] = have;
  s_new[i] = need;
  s_first[i] = first;
  if (i < n) {
    plan[i * kPlanInts] = seq >= 0 ? t : 0;
    plan[i * kPlanInts + 1] = len;
    plan[i * kPlanInts + 2] = next;
  }
  if (seq >= 0) {
    v.meta[2 * seq] = len + t;
    v.meta[2 * seq + 1] = next + t;
  }
  __syncthreads();
  const Spread w(n);
  for (int e = w.first; e < n; e += w.step) {
    const int b = s_list[e];
    if (b < 0) continue;
    for (int j = w.lane; j < s_new[e]; j += w.lanes) {
      const int p = fresh[s_first[e] + j];
      v.ref[p] = 1;
      v.table[static_cast<size_t>(b) * v.width + s_len[e] + j] = p;
    }
  }
}

// kWriteTokens tokens per block, of one (entry, head) or, where calls write few
// tokens (a step's), of several: 1 << span tokens of each. Eight lanes per token,
// each D / 8 values of its key and of its value. Bound by HBM: 8 prompts of up to 2048
// tokens, 32 heads of 128, 0.47 GB in 69 us. (A step of 256 sequences x 32 heads: 14.3
// us with its plan, 22.5 with a block per entry and head.)
constexpr int kWriteTokens = 32;
// 448 / amax overflows below 448 / FLT_MAX (just above 2^-120): such vectors are stored as zero.
constexpr float kTinyVector = 0x1p-119f;

template <int D, bool F8>
__global__ void __launch_bounds__(256)
    write_kernel(PoolView v, int n, const int32_t* __restrict__ seqs,
                 const __nv_bfloat16* __restrict__ K, const __nv_bfloat16* __restrict__ V, int T,
                 int span, const float* __restrict__ score, const int32_t* plan) {
  constexpr int LPT = 8, EPL = D / LPT, NV = EPL / 8;
  const int token = threadIdx.x / LPT, l = threadIdx.x % LPT;
  const int unit = (blockIdx.x * kWriteTokens >> span) + (token >> span);  // (entry, head)
  const int t = blockIdx.y * kWriteTokens + (token & ((1 << span) - 1));
  const int e = unit / v.heads, head = unit - e * v.heads;
  grid_dependency_wait();
  grid_launch_dependents();
  if (e >= n || t >= plan[e * kPlanInts]) return;  // whole groups of eight lanes leave together
  const unsigned gmask = 0xffu << (threadIdx.x & 31 & ~(LPT - 1));
  const int seq = seqs[e], slot = plan[e * kPlanInts + 1] + t;
  const size_t src = (static_cast<size_t>(unit) * T + t) * D + l * EPL;
  uint4 raw[2][NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    raw[0][j] = *reinterpret_cast<const uint4*>(K + src + 8 * j);
    raw[1][j] = *reinterpret_cast<const uint4*>(V + src + 8 * j);
  }
  const int p = held_page(v, seq, slot >> v.shift);
  if (p < 0) return;
  const size_t to = slot_base(v, p, head) + (slot & (v.page - 1));
  if (l == 0) {
    v.pos[to] = plan[e * kPlanInts + 2] + t;
    v.score[(static_cast<size_t>(seq) * v.heads + head) * v.cap + slot] =
        score ? score[static_cast<size_t>(unit) * T + t] : 0.f;
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t* dst = (kv ? v.V : v.K) + to * v.row_bytes;
    if constexpr (F8) {
      float f[EPL];
#pragma unroll
      for (int j = 0; j < NV; ++j) bf16x8_to_f32(raw[kv][j], f + 8 * j);
      // a NaN or an infinity has no code: the vector becomes NaN by its scale
      bool wild = false;
#pragma unroll
      for (int j = 0; j < EPL; ++j) wild |= !(fabsf(f[j]) < INFINITY);
      wild = __ballot_sync(gmask, wild) & gmask;
      if (wild) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) f[j] = 0.f;
      }
      uint32_t pairs[EPL / 2];
      float sc = quantize_e4m3<EPL>(f, gmask, LPT, pairs, kTinyVector);
      if (wild) sc = __int_as_float(0x7fc00000);
      if constexpr (EPL == 16)
        *reinterpret_cast<uint4*>(dst + l * EPL) =
            make_uint4(pairs[0] | (pairs[1] << 16), pairs[2] | (pairs[3] << 16),
                       pairs[4] | (pairs[5] << 16), pairs[6] | (pairs[7] << 16));
      else
        *reinterpret_cast<uint2*>(dst + l * EPL) =
            make_uint2(pairs[0] | (pairs[1] << 16), pairs[2] | (pairs[3] << 16));
      if (l == 0) (kv ? v.vscale : v.kscale)[to] = sc;
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        *reinterpret_cast<uint4*>(dst + (l * EPL + 8 * j) * 2) = raw[kv][j];
    }
  }
}

// ------------------------------------------------------------------ compact
// Scores order as fp32 values do, NaN above all, the two zeros equal.
__device__ __forceinline__ unsigned score_key(float x) {
  if (x != x) return 0xffffffffu;
  const unsigned u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectKeys = 44 * 1024;  // scores whose keys are held in shared memory
constexpr int kDigit = 11;              // bits of a radix step: 3 steps
// Copies of the histogram, by lane: scores crowd in few exponents, and a warp's
// additions to one word run one after the other (78 us for 128 rows of 32768 with
// steps of 8 bits from global memory, 33 us with all this). Bound by these steps and
// the block's barriers between them, not by the row's 4 bytes a token.
constexpr int kHists = 4;

// Blocks (head, entry, layer) select; the block behind the last head of entry 0
// plans its layer (alone in the grid where no sequence can be longer than h + r): plan of an entry = {first fresh page or -1, -, -, -}. The
// selection reads lengths and scores only and the plan writes neither, so the
// two run side by side. where[]: slot (page * page size + offset) of each kept
// token, ascending; kept[]: its score. The h-th largest key is found by an
// MSB-first radix select over keys held in shared memory (a row of up to kSelectKeys
// scores is read from HBM once); then a warp counts, and in a second pass places,
// the kept ones of its contiguous part by votes.
__global__ void __launch_bounds__(kSelectThreads, 2)
    compact_select_kernel(PoolView v0, int n, const int32_t* __restrict__ seqs, int h, int r,
                          int32_t* fresh_all, int fresh_stride, int32_t* plan_all,
                          int32_t* __restrict__ where, float* __restrict__ kept, int held) {
  extern __shared__ unsigned keys[];  // `held` of them
  const PoolView v = at_layer(v0, blockIdx.z);
  const int k = h + r, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int wsum[33];
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y) return;
    __shared__ int s_list[kPlanThreads];
    int32_t* fresh = fresh_all + static_cast<size_t>(blockIdx.z) * fresh_stride;
    int32_t* plan = plan_all + static_cast<size_t>(blockIdx.z) * n * kPlanInts;
    int seq = list_entry(v, seqs, n, s_list);
    if (seq >= 0 && seq_length(v, seq) <= k) seq = -1;
    const int need = seq < 0 ? 0 : pages_of(v, k);
    const int first = take_pages(v, need, fresh, wsum);
    if (seq >= 0 && first < 0) atomicOr(v.err, kErrNoPages);
    if (tid < n) plan[tid * kPlanInts] = seq >= 0 ? first : -1;
    return;
  }
  __shared__ uint4 hist4[1 << kDigit];  // kHists counts a bin
  unsigned* hist = reinterpret_cast<unsigned*>(hist4);
  __shared__ unsigned s_prefix;
  __shared__ int s_rank;
  const int head = blockIdx.x, e = blockIdx.y, seq = seqs[e];
  if (seq < 0 || seq >= v.seqs) return;  // the planning block reports it
  const int T = v.meta[2 * seq];
  if (T <= k || T > v.cap) return;
  const float* cs = v.score + (static_cast<size_t>(seq) * v.heads + head) * v.cap;
  const int n_cand = T - r;
  const bool local = n_cand <= held;
  if (local && h > 0) {
    // four loads in flight per thread: the compiler keeps loads behind shared stores
    for (int p0 = 0; p0 < n_cand; p0 += 16 * kSelectThreads) {
      float4 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = p0 + 4 * (tid + kSelectThreads * i);  // rows are whole pages: 16-byte loads stay inside
        x[i] = p < n_cand ? *reinterpret_cast<const float4*>(cs + p) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int p = p0 + 4 * (tid + kSelectThreads * i);
        if (p < n_cand)
          *reinterpret_cast<uint4*>(keys + p) =
              make_uint4(score_key(x[i].x), score_key(x[i].y), score_key(x[i].z), score_key(x[i].w));
      }
    }
  }
  auto key = [&](int p) { return local ? keys[p] : score_key(cs[p]); };
  // Keep candidate p iff its key is above tau, or equals tau and p is not
  // among the first `skip` candidates of that key.
  unsigned tau = 0xffffffffu;
  int skip = 0x7fffffff;
  if (h > 0) {
    unsigned prefix = 0, mask = 0;
    int rank = n_cand - h;
    for (int shift = 32 - kDigit; mask != 0xffffffffu; shift -= kDigit) {
      const int s = max(shift, 0), bits = shift < 0 ? kDigit + shift : kDigit;
      const unsigned low = (1u << bits) - 1;
      for (int i = tid; i < 1 << kDigit; i += kSelectThreads) hist4[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      // (one addition for all lanes of a bin, found by a match, took 10 us longer)
#pragma unroll 4
      for (int p = tid; p < n_cand; p += kSelectThreads) {
        const unsigned u = key(p);
        if ((u & mask) == prefix) atomicAdd(&hist[((u >> s) & low) * kHists + (lane & (kHists - 1))], 1u);
      }
      __syncthreads();
      // the bin of the rank-th key: two bins a thread, one block scan
      const uint4 x = hist4[2 * tid], y = hist4[2 * tid + 1];
      const int a = static_cast<int>(x.x + x.y + x.z + x.w), b = static_cast<int>(y.x + y.y + y.z + y.w);
      int total;
      const int before = block_exclusive_scan(a + b, wsum, &total);
      if (before <= rank && rank < before + a + b) {
        const bool second = rank >= before + a;
        s_prefix = prefix | (static_cast<unsigned>(2 * tid + second) << s);
        s_rank = rank - before - (second ? a : 0);
      }
      __syncthreads();
      prefix = s_prefix;
      rank = s_rank;
      mask |= low << s;
    }
    tau = prefix;
    skip = rank;
  }
  // a warp's part: whole groups of 32 candidates, counted above and at tau
  const int groups = (T + 31) / 32, per = (groups + kSelectWarps - 1) / kSelectWarps;
  const int g0 = min(groups, warp * per), g1 = min(groups, g0 + per);
  int above = 0, equal = 0;  // above: kept whatever the ties are
#pragma unroll 4
  for (int g = g0; g < g1; ++g) {
    const int p = 32 * g + lane;
    const bool cand = p < n_cand && h > 0;
    const unsigned u = cand ? key(p) : 0u;
    above += __popc(__ballot_sync(0xffffffffu, cand ? u > tau : p >= n_cand && p < T));
    equal += __popc(__ballot_sync(0xffffffffu, cand && u == tau));
  }
  int dummy;
  const int eq0 = __shfl_sync(0xffffffffu, block_exclusive_scan(lane ? 0 : equal, wsum, &dummy), 0);
  const int ties = max(0, eq0 + equal - max(skip, eq0));  // of this part, those past the skipped
  int at = __shfl_sync(0xffffffffu, block_exclusive_scan(lane ? 0 : above + ties, wsum, &dummy), 0);
  const size_t out = ((static_cast<size_t>(blockIdx.z) * n + e) * v.heads + head) * k;
  const unsigned below = (1u << lane) - 1;
  int eq = eq0;
  for (int g = g0; g < g1; g += 4) {  // four groups at a time, their loads in flight together
    int slot[4], page[4];
    float value[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = 32 * (g + i) + lane;
      const bool in = g + i < g1, cand = in && p < n_cand && h > 0;
      const unsigned u = cand ? key(p) : 0u;
      const unsigned same = __ballot_sync(0xffffffffu, cand && u == tau);
      const bool keep = cand ? u > tau || (u == tau && eq + __popc(same & below) >= skip)
                             : in && p >= n_cand && p < T;
      const unsigned all = __ballot_sync(0xffffffffu, keep);
      slot[i] = keep ? at + __popc(all & below) : -1;
      at += __popc(all);
      eq += __popc(same);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = 32 * (g + i) + lane;
      page[i] = slot[i] < 0 ? 0 : v.table[static_cast<size_t>(seq) * v.width + (p >> v.shift)];
      value[i] = slot[i] < 0 ? 0.f : cs[p];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = 32 * (g + i) + lane;
      if (slot[i] < 0) continue;
      const bool held_one = page[i] >= 0 && page[i] < v.pages;
      if (!held_one) atomicOr(v.err, kErrBadState);
      where[out + slot[i]] = held_one ? (page[i] << v.shift) + (p & (v.page - 1)) : -1;
      kept[out + slot[i]] = value[i];
    }
  }
}

// One warp per 1 KB of keys of a head's kept slots: all loads of a lane are in flight
// before its stores (2 KB a warp: 145 against 135 us with the case below; four slots of
// codes a warp, half the bytes: 42 against 40 us for 8 prompts to 460 tokens). Bound by
// HBM: 4096 of 32768 tokens of 128 heads, 0.54 GB in 86 us. The first block of an entry
// also puts the new pages in the table and drops the old ones, which the gather does
// not read again.
constexpr int gather_slots(int row) { return 1024 / row; }

template <int ROW>
__global__ void __launch_bounds__(256)
    compact_gather_kernel(PoolView v0, int n, const int32_t* __restrict__ seqs, int k,
                          const int32_t* fresh_all, int fresh_stride,
                          const int32_t* plan_all, const int32_t* where,
                          const float* kept) {
  constexpr int SLOTS = gather_slots(ROW);
  constexpr int CH = ROW / 16;                     // 16-byte chunks of a vector
  constexpr int PER = 2 * CH;                      // chunks of a slot: key, then value
  constexpr int NC = (PER * SLOTS + 31) / 32;    // chunks per lane
  const PoolView v = at_layer(v0, blockIdx.z);
  const int e = blockIdx.x / v.heads, head = blockIdx.x % v.heads;
  grid_dependency_wait();
  grid_launch_dependents();
  const int first = plan_all[(static_cast<size_t>(blockIdx.z) * n + e) * kPlanInts];
  if (first < 0) return;
  const int32_t* fresh = fresh_all + static_cast<size_t>(blockIdx.z) * fresh_stride + first;
  const int seq = seqs[e], lane = threadIdx.x & 31;
  if (blockIdx.y == 0 && head == 0) {
    const int old = pages_of(v, v.meta[2 * seq]), now = pages_of(v, k);
    for (int j = threadIdx.x; j < old; j += blockDim.x) {
      int32_t* t = v.table + static_cast<size_t>(seq) * v.width + j;
      const int p = *t;
      if (p >= 0 && p < v.pages) drop_page(v, p);
      *t = j < now ? fresh[j] : -1;
    }
    for (int j = threadIdx.x; j < now; j += blockDim.x) v.ref[fresh[j]] = 1;
    __syncthreads();
    if (threadIdx.x == 0) v.meta[2 * seq] = k;
  }
  const size_t in = ((static_cast<size_t>(blockIdx.z) * n + e) * v.heads + head) * k;
  const int slot0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * SLOTS;
  uint4 x[NC];
  uint8_t* dst[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = lane + 32 * i, slot = slot0 + c / PER;
    dst[i] = nullptr;
    if (c >= PER * SLOTS || slot >= k) continue;
    const int w = where[in + slot];
    if (w < 0) continue;
    const int at = c % PER, kv = at >= CH, byte = (kv ? at - CH : at) * 16;
    const size_t from = slot_base(v, w >> v.shift, head) + (w & (v.page - 1));
    const size_t to = slot_base(v, fresh[slot >> v.shift], head) + (slot & (v.page - 1));
    x[i] = *reinterpret_cast<const uint4*>((kv ? v.V : v.K) + from * ROW + byte);
    dst[i] = (kv ? v.V : v.K) + to * ROW + byte;
  }
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (dst[i]) *reinterpret_cast<uint4*>(dst[i]) = x[i];
  const int slot = slot0 + lane;
  if (lane < SLOTS && slot < k) {
    v.score[(static_cast<size_t>(seq) * v.heads + head) * v.cap + slot] = kept[in + slot];
    const int w = where[in + slot];
    if (w >= 0) {
      const size_t from = slot_base(v, w >> v.shift, head) + (w & (v.page - 1));
      const size_t to = slot_base(v, fresh[slot >> v.shift], head) + (slot & (v.page - 1));
      v.pos[to] = v.pos[from];
      if (v.kscale) {
        v.kscale[to] = v.kscale[from];
        v.vscale[to] = v.vscale[from];
      }
    }
  }
}

}  // namespace

cudaError_t pool_fork(const PoolView& v, int layers, int n, const int32_t* src, const int32_t* dst,
                      bool share, int32_t* fresh, int32_t* plan, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  cudaError_t e = launch_after(fork_plan_kernel, dim3(layers), kPlanThreads, 0, stream, v, n, src, dst,
                               share, fresh, share ? n : n * v.width, plan);
  if (e != cudaSuccess) return e;
  // slabs of kSlab slots, or longer ones where those of full sequences would be more than some 4
  // blocks an SM (32 where each has pages to copy): most of what the sequences could hold may be
  // empty, and a pool 40 times as wide as its contents then took 271 us for 202. (4 against 12
  // and 24: 4 beams in a pool of 32768 tokens a sequence 9.9, 10.0, 11.5 us, 4 full ones 15.6, 16.1, 16.9)
  const int units = n * v.heads, most = (share ? 4 : 32) * num_sms();
  const bool many = static_cast<int64_t>(units) * layers >= kManySlabs;
  const int x = many ? (units + 7) / 8 : units, slabs = (v.cap + kSlab - 1) / kSlab;
  const int y = static_cast<int>(std::min<int64_t>(slabs, 1 + most / (static_cast<int64_t>(x) * layers)));
  const int slab = (slabs + y - 1) / y * kSlab;
  return launch_after(many ? fork_copy_kernel<32> : fork_copy_kernel<256>, dim3(x, y, layers), 256, 0,
                      stream, v, n, src, dst, share, slab, static_cast<const int32_t*>(plan));
}

cudaError_t pool_free(const PoolView& v, int layers, int n, const int32_t* seqs,
                      cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  return launch_after(free_kernel, dim3(layers), kPlanThreads, 0, stream, v, n, seqs);
}

cudaError_t pool_write(const PoolView& v, int n, const int32_t* seqs, const void* K, const void* V,
                       int T, const int32_t* lens, const float* score, int32_t* fresh,
                       int32_t* plan, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  cudaError_t e =
      launch_after(write_plan_kernel, dim3(1), kPlanThreads, 0, stream, v, n, seqs, T, lens, fresh, plan);
  if (e != cudaSuccess || T == 0) return e;
  int span = 0;
  while (1 << span < kWriteTokens && 1 << span < T) ++span;
  const int units = kWriteTokens >> span;  // per block
  const dim3 grid((n * v.heads + units - 1) / units, (T + kWriteTokens - 1) / kWriteTokens);
  auto kk = static_cast<const __nv_bfloat16*>(K);
  auto vv = static_cast<const __nv_bfloat16*>(V);
  auto kern = v.d == 128 ? (v.kscale ? write_kernel<128, true> : write_kernel<128, false>)
                         : (v.kscale ? write_kernel<64, true> : write_kernel<64, false>);
  return launch_after(kern, grid, 256, 0, stream, v, n, seqs, kk, vv, T, span, score,
                      static_cast<const int32_t*>(plan));
}

cudaError_t pool_compact(const PoolView& v, int layers, int n, const int32_t* seqs, int h, int r,
                         int32_t* fresh, int32_t* plan, int32_t* where, float* kept,
                         cudaStream_t stream) {
  const int k = h + r;
  if (n == 0) return cudaSuccess;
  const int stride = n * ((k + v.page - 1) >> v.shift);
  // the keys of a row in shared memory, where rows can be that long
  const bool any = k < v.cap;  // else no sequence can be longer than h + r, and the list is checked alone
  const int held = any ? std::min(v.cap, kSelectKeys) : 0;
  static int opted_in[kMaxDevices] = {};
  cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(compact_select_kernel),
                                   kSelectKeys * sizeof(unsigned), opted_in);
  if (e != cudaSuccess) return e;
  e = launch_after(compact_select_kernel, any ? dim3(v.heads + 1, n, layers) : dim3(1, 1, layers), kSelectThreads,
                   held * sizeof(unsigned), stream, v, n, seqs, h, r, fresh, stride, plan, where, kept, held);
  if (e != cudaSuccess || !any) return e;
  const int slots = 8 * gather_slots(v.row_bytes);  // per block
  const dim3 grid(n * v.heads, (k + slots - 1) / slots, layers);
  auto kern = v.row_bytes == 256 ? compact_gather_kernel<256>
              : v.row_bytes == 128 ? compact_gather_kernel<128> : compact_gather_kernel<64>;
  return launch_after(kern, grid, 256, 0, stream, v, n, seqs, k, static_cast<const int32_t*>(fresh),
                      stride, static_cast<const int32_t*>(plan), static_cast<const int32_t*>(where),
                      static_cast<const float*>(kept));
}

}  // namespace h2o
