// Attention of single tokens over the paged cache: a prefix that the whole
// batch shares, then each sequence's own tokens, in the plainest form. For row
// (b, query head) with key head h: s_j = q . k_j / sqrt(d), lse = log sum_j
// exp(s_j), p_j = exp(s_j - lse), out = sum_j p_j v_j; the scores of the
// sequence's slots grow by the probabilities of the head's group, those of the
// prefix by the sum over the batch.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pool.h"

namespace h2o {
namespace {

constexpr int kThreads = 128;

// Row b's sequence, or -1 (no work, or reported).
__device__ int row_seq(const AttendArgs& a, int b) {
  const int s = a.seqs[b];
  if (s == -1) return -1;
  bool bad = s < 0 || s >= a.v.seqs || s == a.prefix;
  for (int j = 0; j < b; ++j) bad |= a.seqs[j] == s;
  if (bad) atomicOr(a.v.err, kErrBadList);
  return bad ? -1 : s;
}

__device__ int length_of(const PoolView& v, int s) {
  if (s < 0) return 0;
  const int n = v.meta[2 * s];
  if (n >= 0 && n <= v.cap) return n;
  atomicOr(v.err, kErrBadState);
  return 0;
}

// Slot of token j of the prefix (j < P) or of sequence s, or -1.
__device__ long slot_of(const AttendArgs& a, int s, int P, int j, int head) {
  const PoolView& v = a.v;
  const int seq = j < P ? a.prefix : s, t = j < P ? j : j - P;
  const int p = v.table[static_cast<size_t>(seq) * v.width + (t >> v.shift)];
  if (p < 0 || p >= v.pages) {
    atomicOr(v.err, kErrBadState);
    return -1;
  }
  return ((static_cast<long>(p) * v.heads + head) << v.shift) + (t & (v.page - 1));
}

__device__ float stored(const PoolView& v, bool val, long slot, int c) {
  const uint8_t* base = (val ? v.V : v.K) + slot * v.row_bytes;
  if (!v.kscale) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[c]);
  const __half_raw h = __nv_cvt_fp8_to_halfraw(base[c], __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h)) * (val ? v.vscale : v.kscale)[slot];
}

// One block per (b, query head); logits in scratch [b][query head][2 cap].
__global__ void __launch_bounds__(kThreads)
    attend_rows_kernel(const AttendArgs a, float* logits, float* lse2) {
  const PoolView& v = a.v;
  const int hq = v.heads * a.group, b = blockIdx.x / hq, head = blockIdx.x % hq / a.group;
  const int s = row_seq(a, b);
  if (s < 0) return;
  const int P = length_of(v, a.prefix), n = P + length_of(v, s);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + static_cast<size_t>(blockIdx.x) * v.d;
  float* L = logits + static_cast<size_t>(blockIdx.x) * 2 * v.cap;
  __shared__ float red[kThreads];
  const int tid = threadIdx.x;
  const float qs = kLog2e / sqrtf(static_cast<float>(v.d));
  float m = -INFINITY;
  for (int j = tid; j < n; j += kThreads) {
    const long at = slot_of(a, s, P, j, head);
    float x = 0.f;
    if (at >= 0)
      for (int c = 0; c < v.d; ++c) x = fmaf(__bfloat162float(q[c]), stored(v, false, at, c), x);
    L[j] = x * qs;
    m = fmaxf(m, L[j]);
  }
  red[tid] = m;
  __syncthreads();
  for (int i = 0; i < kThreads; ++i) m = fmaxf(m, red[i]);
  __syncthreads();
  float l = 0.f;
  for (int j = tid; j < n; j += kThreads) l += exp2f(L[j] - m);
  red[tid] = l;
  __syncthreads();
  l = 0.f;
  for (int i = 0; i < kThreads; ++i) l += red[i];
  const float lse = n ? m + log2f(l) : -INFINITY;
  if (tid == 0) {
    lse2[blockIdx.x] = lse;
    if (a.lse) a.lse[blockIdx.x] = n ? lse / kLog2e : -INFINITY;
  }
  if (tid < v.d) {
    float o = 0.f;
    for (int j = 0; j < n; ++j) {
      const long at = slot_of(a, s, P, j, head);
      if (at >= 0) o = fmaf(exp2f(L[j] - lse), stored(v, true, at, tid), o);
    }
    static_cast<__nv_bfloat16*>(a.out)[static_cast<size_t>(blockIdx.x) * v.d + tid] = __float2bfloat16(o);
  }
}

// Block (key head, b), b == n: the prefix.
__global__ void __launch_bounds__(kThreads)
    attend_score_kernel(const AttendArgs a, const float* logits, const float* lse2) {
  const PoolView& v = a.v;
  const int head = blockIdx.x, b = blockIdx.y, P = length_of(v, a.prefix);
  const int s = b < a.n ? row_seq(a, b) : a.prefix;
  if (s < 0) return;
  const int n = length_of(v, s);
  for (int j = threadIdx.x; j < n; j += kThreads) {
    float sum = 0.f;
    for (int i = b < a.n ? b : 0; i < (b < a.n ? b + 1 : a.n); ++i) {
      if (b == a.n && row_seq(a, i) < 0) continue;
      for (int g = 0; g < a.group; ++g) {
        const size_t row = (static_cast<size_t>(i) * v.heads + head) * a.group + g;
        sum += exp2f(logits[row * 2 * v.cap + (b < a.n ? P + j : j)] - lse2[row]);
      }
    }
    v.score[(static_cast<size_t>(s) * v.heads + head) * v.cap + j] += sum;
  }
}

}  // namespace

size_t pool_attend_simple_scratch(const AttendArgs& a) {
  return static_cast<size_t>(a.n) * a.v.heads * a.group * (2 * static_cast<size_t>(a.v.cap) + 1) * 4;
}

cudaError_t pool_attend_simple(const AttendArgs& a, void* scratch, cudaStream_t stream) {
  const size_t rows = static_cast<size_t>(a.n) * a.v.heads * a.group;
  if (rows == 0) return cudaSuccess;
  float* logits = static_cast<float*>(scratch);
  float* lse2 = logits + rows * 2 * a.v.cap;
  attend_rows_kernel<<<static_cast<unsigned>(rows), kThreads, 0, stream>>>(a, logits, lse2);
  if (a.accumulate)
    attend_score_kernel<<<dim3(a.v.heads, a.n + (a.prefix >= 0)), kThreads, 0, stream>>>(a, logits, lse2);
  return cudaGetLastError();
}

}  // namespace h2o
