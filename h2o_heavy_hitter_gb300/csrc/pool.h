// Host-side launchers of the paged cache (h2o_pool_*). Plain C++ types only;
// every launcher enqueues on `stream` and returns the launch status.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace h2o {

// The arrays of a pool from one layer on, and its sizes. A layer's arrays lie
// one after the other: element (layer, ...) of an array is at layer * (the
// array's size per layer).
struct PoolView {
  uint8_t* K;       // [layers][pages][heads][page][d] bf16 or E4M3 codes
  uint8_t* V;
  float* kscale;    // [layers][pages][heads][page], E4M3 pool only (else null)
  float* vscale;
  int32_t* pos;     // [layers][pages][heads][page] token position of a slot
  float* score;     // [layers][seqs][heads][cap] accumulated score by sequence
  int32_t* table;   // [layers][seqs][width] pages of a sequence, -1 behind the last
  int32_t* meta;    // [layers][seqs][2] {length, next position}
  int32_t* ref;     // [layers][pages] sequences that hold a page
  int32_t* err;     // device error word
  int pages, seqs, width, heads, d;
  int page, shift;  // tokens per page = 1 << shift
  int cap;          // width * page, the longest sequence
  int row_bytes;    // bytes of one stored key or value vector
};

constexpr int kPoolMaxList = 1024;  // longest list of sequences of one call: one thread each
constexpr int kPoolMaxGroup = 32;   // query heads per key head: the own rows of a sequence fit one warp

// Fresh pages are found by one block per layer ("plan"), which fork, copy and write
// let change the tables too; a second kernel then moves the tokens. `fresh` (scratch)
// has room for every page the call can ask for, per layer; `plan` (scratch) for
// kPlanInts ints per layer and list entry.
constexpr int kPlanInts = 4;

// Sequence dst[i] becomes a copy of src[i]: whole pages shared and the partial
// last page copied (share), or every page copied. fresh: n (share) or n * width.
cudaError_t pool_fork(const PoolView& v, int layers, int n, const int32_t* src, const int32_t* dst,
                      bool share, int32_t* fresh, int32_t* plan, cudaStream_t stream);
cudaError_t pool_free(const PoolView& v, int layers, int n, const int32_t* seqs,
                      cudaStream_t stream);
// Appends lens[i] (or T) tokens to sequence seqs[i] of one layer (T = 0: the list is checked
// alone). fresh: n * ceil(T / page).
cudaError_t pool_write(const PoolView& v, int n, const int32_t* seqs, const void* K, const void* V,
                       int T, const int32_t* lens, const float* score, int32_t* fresh,
                       int32_t* plan, cudaStream_t stream);

// Keeps the r last tokens and the h others of largest (score, slot) of every
// head of each sequence longer than h + r. fresh: n * ceil(k / page) per layer;
// where / kept: layers * n * heads * k. With h + r >= cap (none of the three is then
// needed) it checks the list alone.
cudaError_t pool_compact(const PoolView& v, int layers, int n, const int32_t* seqs, int h, int r,
                         int32_t* fresh, int32_t* plan, int32_t* where, float* kept,
                         cudaStream_t stream);

// Attention of one token of each sequence of a batch (pool_attend.cu).
struct AttendArgs {
  PoolView v;            // of the layer
  const int32_t* seqs;   // [n]
  int n;
  int before;            // entries of the caller's list ahead of seqs, whose sequences are named already
  int prefix;            // sequence whose tokens every row attends to first, or -1
  int group;             // query heads per key head
  const void* q;         // bf16 [n][heads * group][d]
  void* out;             // bf16 [n][heads * group][d]
  float* lse;            // [n][heads * group], natural log; may be null
  int accumulate;        // add the probabilities to the scores
  const CUtensorMap* kmap;  // host: the layer's keys and values (pool_page_map)
  const CUtensorMap* vmap;
};
// Tensor map of a layer's keys or values in boxes of a page's tokens x 64
// channels (bf16, 128-byte swizzle) or x all codes (E4M3; keys swizzled by d bytes).
cudaError_t pool_page_map(CUtensorMap* m, const PoolView& v, bool keys);
size_t pool_attend_scratch(const AttendArgs& a);
cudaError_t pool_attend(const AttendArgs& a, void* scratch, cudaStream_t stream);
}  // namespace h2o
