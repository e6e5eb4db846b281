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
  int32_t* refused; // [layers][seqs] kRefused bits of a sequence's last write or append
  int32_t* err;     // device error word
  int pages, seqs, width, heads, d;
  int page, shift;  // tokens per page = 1 << shift
  int cap;          // width * page, the longest sequence
  int row_bytes;    // bytes of one stored key or value vector
};

// A sequence's tokens of its last write or append were refused: its last tokens are no drafts, and
// (kRefusedQueries) there are no queries either. Only a call that is served, or ends the round, takes these away.
constexpr int kRefused = 1, kRefusedQueries = 2;

constexpr int kPoolMaxList = 1024;  // longest list of sequences of one call: one thread each
// 448 / amax overflows below 448 / FLT_MAX (just above 2^-120): such vectors are stored as zero.
constexpr float kTinyVector = 0x1p-119f;
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

// The plan of a write alone: pages, lengths and (unless the tokens are drafts) next positions; plan of an
// entry = {tokens to write (0: none), first slot, next position before, -}. mark: kRefused bits of what is refused.
cudaError_t pool_write_plan(const PoolView& v, int n, const int32_t* seqs, int T, const int32_t* lens,
                            bool drafts, int mark, int32_t* fresh, int32_t* plan, cudaStream_t stream);

// Keeps the r last tokens and the h others of largest (score, slot) of every
// head of each sequence longer than h + r. fresh: n * ceil(k / page) per layer;
// where / kept: layers * n * heads * k. With h + r >= cap (none of the three is then
// needed) it checks the list alone.
cudaError_t pool_compact(const PoolView& v, int layers, int n, const int32_t* seqs, int h, int r,
                         int32_t* fresh, int32_t* plan, int32_t* where, float* kept,
                         cudaStream_t stream);

// Of the last lens[i] (or T) tokens of each sequence, keeps those that path [n][P] names, in order. plan:
// kAcceptInts ints per layer and entry. rows, tiles (null: none), n + 1 ints each, and list, n P ints, are for
// pool_accept_scores.
constexpr int kAcceptInts = 8;
constexpr int kScoreKeys = 128;  // keys of a block of pool_accept_scores
cudaError_t pool_accept(const PoolView& v, int layers, int n, const int32_t* seqs, int T, const int32_t* lens,
                        const int32_t* path, int P, int prefix, int32_t* plan, int32_t* rows, int32_t* tiles,
                        int32_t* list, cudaStream_t stream);

// Adds the probabilities exp(q . k / sqrt(d) - lse) of the drafts that pool_accept kept, rows of q
// [n][T][heads * group][d] and lse [n][T][heads * group], to the scores of the tokens that they attend to.
struct AcceptArgs {
  PoolView v;  // of the layer
  const int32_t* seqs;
  int n, prefix, group;
  const void* q;
  const float* lse;
  const int32_t *plan, *rows, *tiles, *list;
};
cudaError_t pool_accept_scores(const AcceptArgs& a, cudaStream_t stream);

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
// The drafts of a call on a tree: a.seqs is the list of n sequences, a.n = n * T the rows of queries a head.
struct TreeArgs {
  int n, T;
  const int32_t* lens;    // [n] drafts of an entry (null: T)
  const int32_t* parent;  // [n][T] (null: a chain)
};
size_t pool_tree_scratch(const AttendArgs& a, const TreeArgs& t);
cudaError_t pool_tree(const AttendArgs& a, const TreeArgs& t, void* scratch, cudaStream_t stream);

// Tensor map of a layer's keys or values in boxes of a page's tokens x 64
// channels (bf16, 128-byte swizzle) or x all codes (E4M3; keys swizzled by d bytes).
cudaError_t pool_page_map(CUtensorMap* m, const PoolView& v, bool keys);
size_t pool_attend_scratch(const AttendArgs& a);
cudaError_t pool_attend(const AttendArgs& a, void* scratch, cudaStream_t stream);
}  // namespace h2o
