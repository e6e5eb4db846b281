// Block-wide scan and radix-select step shared by the selection kernels.
#pragma once

namespace h2o {

// Block-wide exclusive scan of one int per thread; *total gets the sum.
// wsum: 33 ints of shared memory.
__device__ __forceinline__ int block_exclusive_scan(int x, int* wsum, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nw = blockDim.x >> 5;
  int incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int v = lane < nw ? wsum[lane] : 0;
    int vi = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, vi, off);
      if (lane >= off) vi += y;
    }
    wsum[lane] = vi - v;
    if (lane == 31) wsum[32] = vi;
  }
  __syncthreads();
  const int r = wsum[warp] + incl - x;
  *total = wsum[32];
  __syncthreads();
  return r;
}

// One step of an MSB-first radix select: warp 0 finds the bin of hist[256] that
// holds the rank-th key in ascending order. Each lane sums eight bins, a
// shuffle scan places the lanes, and the one lane whose range contains the
// rank walks its eight bins and writes the extended prefix and the rank within
// the bin. Between block barriers.
__device__ __forceinline__ void radix_pick(const unsigned* hist, int rank, unsigned prefix,
                                           int shift, unsigned* s_prefix, int* s_rank) {
  const int tid = threadIdx.x;
  if (tid >= 32) return;
  unsigned c[8];
  int local = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] = hist[tid * 8 + j];
    local += static_cast<int>(c[j]);
  }
  int incl = local;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, off);
    if (tid >= off) incl += y;
  }
  int cum = incl - local;
  if (cum <= rank && rank < incl) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (cum + static_cast<int>(c[j]) > rank) {
        *s_prefix = prefix | (static_cast<unsigned>(tid * 8 + j) << shift);
        *s_rank = rank - cum;
        break;
      }
      cum += static_cast<int>(c[j]);
    }
  }
}

}  // namespace h2o
