// C ABI of the paged cache (h2o_pool_*, declared in include/h2o.h). Host side
// only: argument checks, the pool's memory, scratch and launches on the current
// PyTorch stream.
#include <c10/cuda/CUDAFunctions.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <memory>
#include <new>
#include <string>
#include <vector>

#include "h2o.h"
#include "host.h"
#include "pool.h"
#include "rotary.h"

using namespace h2o::host;

struct h2o_pool {
  int layers = 0;
  int device = 0;
  int kv_format = 0;
  void* base = nullptr;  // single allocation
  h2o::PoolView v{};     // layer 0
  std::vector<CUtensorMap> maps;  // keys and values of every layer
};

namespace {

size_t slots_per_layer(const h2o::PoolView& v) {
  return static_cast<size_t>(v.pages) * v.heads * v.page;
}

h2o::PoolView layer_view(const h2o_pool* p, int layer) {
  h2o::PoolView v = p->v;
  const size_t l = layer, slots = slots_per_layer(v) * l;
  v.K += slots * v.row_bytes;
  v.V += slots * v.row_bytes;
  if (v.kscale) {
    v.kscale += slots;
    v.vscale += slots;
  }
  v.pos += slots;
  v.score += l * v.seqs * v.heads * v.cap;
  v.table += l * v.seqs * v.width;
  v.meta += l * v.seqs * 2;
  v.ref += l * v.pages;
  v.refused += l * v.seqs;
  return v;
}

int check_pool(const h2o_pool* p) {
  if (!p) return fail(H2O_EINVAL, "null pool");
  int cur = -1;
  cudaError_t e = cudaGetDevice(&cur);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (cur != p->device)
    return fail(H2O_EINVAL, "the pool belongs to device " + std::to_string(p->device) +
                                " but device " + std::to_string(cur) + " is current");
  return H2O_OK;
}

// Arguments common to the list operations: n entries, layer >= 0 or, where
// `all` layers can be meant, -1.
int check_list(const h2o_pool* p, int layer, bool all, int n, const void* list) {
  if (!p) return fail(H2O_EINVAL, "null pool");
  if (layer < (all ? -1 : 0) || layer >= p->layers) return fail(H2O_EINVAL, "layer out of range");
  if (n < 0 || n > H2O_POOL_MAX_LIST)
    return fail(H2O_EINVAL, "n must be in [0, H2O_POOL_MAX_LIST]");
  if (n > 0 && !list) return fail(H2O_EINVAL, "null sequence list");
  return check_pool(p);
}

int fork_or_copy(h2o_pool* p, int layer, int n, const int32_t* src, const int32_t* dst,
                 bool share) {
  if (int rc = check_list(p, layer, true, n, src)) return rc;
  if (n > 0 && !dst) return fail(H2O_EINVAL, "null sequence list");
  if (n == 0) return H2O_OK;
  return guarded([&] {
    const h2o::PoolView v = layer_view(p, layer < 0 ? 0 : layer);
    const size_t L = layer < 0 ? p->layers : 1, N = n;
    const size_t fresh = L * N * (share ? 1 : v.width), plan = L * N * h2o::kPlanInts;
    cudaStream_t s = current_stream();
    Scratch mem((fresh + plan) * sizeof(int32_t), s);
    int32_t* m = static_cast<int32_t*>(mem.p);
    return launch_status(h2o::pool_fork(v, static_cast<int>(L), n, src, dst, share, m, m + fresh, s),
                         "pool fork launch");
  });
}

}  // namespace

extern "C" {

int h2o_pool_create(int layers, int pages, int page_size, int heads, int head_dim, int sequences,
                    int max_pages, int kv_format, h2o_pool** out) {
  if (!out) return fail(H2O_EINVAL, "null output pointer");
  *out = nullptr;
  if (kv_format != H2O_KV_BF16 && kv_format != H2O_KV_FP8)
    return fail(H2O_EINVAL, "kv_format must be H2O_KV_BF16 or H2O_KV_FP8");
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return fail(H2O_EINVAL, "page_size must be 16, 32, 64 or 128");
  if (head_dim != 64 && head_dim != 128) return fail(H2O_EINVAL, "head_dim must be 64 or 128");
  if (layers < 1 || layers > 65535) return fail(H2O_EINVAL, "layers out of range");
  if (heads < 1 || heads > H2O_POOL_MAX_HEADS) return fail(H2O_EINVAL, "heads out of range");
  if (pages < 1 || sequences < 1 || sequences > (1 << 20) || max_pages < 1)
    return fail(H2O_EINVAL, "pages, sequences and max_pages must be in range");
  if (static_cast<int64_t>(pages) * heads * page_size >= (int64_t{1} << 31))
    return fail(H2O_EINVAL, "pages * heads * page_size must be below 2^31 (slots of a layer)");
  if (static_cast<int64_t>(max_pages) * page_size > H2O_MAX_T)
    return fail(H2O_EINVAL, "max_pages * page_size exceeds H2O_MAX_T");
  // what the sizes below are made of; 2^56 bytes are more than any device has
  const double want = static_cast<double>(layers) *
                      (static_cast<double>(pages) * heads * page_size * (4 * head_dim + 12) +
                       static_cast<double>(sequences) * max_pages * (4.0 * heads * page_size + 4));
  if (want > 7e16) return fail(H2O_ENOMEM, "pool too large");
  auto* p = new (std::nothrow) h2o_pool();
  if (!p) return fail(H2O_ENOMEM, "out of host memory");
  try {
    p->device = c10::cuda::current_device();
  } catch (const std::exception& ex) {
    delete p;
    return fail(H2O_ECUDA, std::string("no CUDA device: ") + ex.what());
  }
  p->layers = layers;
  p->kv_format = kv_format;
  h2o::PoolView& v = p->v;
  v.pages = pages;
  v.seqs = sequences;
  v.width = max_pages;
  v.heads = heads;
  v.d = head_dim;
  v.page = page_size;
  v.shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  v.cap = max_pages * page_size;
  v.row_bytes = head_dim * (kv_format == H2O_KV_FP8 ? 1 : 2);
  const size_t L = layers, slots = L * slots_per_layer(v);
  const size_t kv = align_up(slots * v.row_bytes, 256);
  const size_t per_slot = align_up(slots * 4, 256);
  const size_t scale = kv_format == H2O_KV_FP8 ? per_slot : 0;
  const size_t score = align_up(L * sequences * heads * v.cap * 4, 256);
  const size_t table = align_up(L * sequences * max_pages * 4, 256);
  const size_t meta = align_up(L * sequences * 8, 256);
  const size_t ref = align_up(L * pages * 4, 256);
  const size_t refused = align_up(L * sequences * 4, 256);
  const size_t total = 2 * kv + per_slot + 2 * scale + score + table + meta + ref + refused + 256;
  cudaStream_t s = nullptr;
  try {
    s = current_stream();
    p->base = device_alloc(total, s);
  } catch (const std::exception& ex) {
    delete p;
    return fail(H2O_ENOMEM, std::string("pool allocation failed: ") + ex.what());
  }
  uint8_t* at = static_cast<uint8_t*>(p->base);
  auto take = [&](size_t bytes) {
    uint8_t* x = at;
    at += bytes;
    return x;
  };
  v.K = take(kv);
  v.V = take(kv);
  if (scale) {
    v.kscale = reinterpret_cast<float*>(take(scale));
    v.vscale = reinterpret_cast<float*>(take(scale));
  }
  v.score = reinterpret_cast<float*>(take(score));
  v.meta = reinterpret_cast<int32_t*>(take(meta));
  v.ref = reinterpret_cast<int32_t*>(take(ref));
  v.refused = reinterpret_cast<int32_t*>(take(refused));
  v.err = reinterpret_cast<int32_t*>(take(256));
  // everything above starts at zero, the two below at -1
  const size_t zeros = static_cast<size_t>(at - static_cast<uint8_t*>(p->base));
  v.pos = reinterpret_cast<int32_t*>(take(per_slot));
  v.table = reinterpret_cast<int32_t*>(take(table));
  cudaError_t e = cudaMemsetAsync(p->base, 0, zeros, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(v.pos, 0xff, per_slot + table, s);
  try {
    p->maps.resize(2 * L);
  } catch (const std::exception&) {
    h2o_pool_destroy(p);
    return fail(H2O_ENOMEM, "out of host memory");
  }
  for (int l = 0; l < layers && e == cudaSuccess; ++l) {
    const h2o::PoolView x = layer_view(p, l);
    e = h2o::pool_page_map(&p->maps[2 * l], x, true);
    if (e == cudaSuccess) e = h2o::pool_page_map(&p->maps[2 * l + 1], x, false);
  }
  if (e != cudaSuccess) {
    h2o_pool_destroy(p);
    return cuda_fail(e, "pool initialisation");
  }
  *out = p;
  return H2O_OK;
}

void h2o_pool_destroy(h2o_pool* p) {
  if (!p) return;
  if (p->base) {
    int cur = -1;
    const bool other = cudaGetDevice(&cur) == cudaSuccess && cur != p->device;
    if (other) cudaSetDevice(p->device);
    guarded([&] {
      // whichever streams its calls ran on; a synchronisation would spoil a capture
      cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
      cudaStreamIsCapturing(current_stream(), &capture);
      if (capture == cudaStreamCaptureStatusNone) cudaDeviceSynchronize();
      device_free(p->base);
      return H2O_OK;
    });
    if (other) cudaSetDevice(cur);
  }
  delete p;
}

int h2o_pool_view(h2o_pool* p, int layer, void** K, void** V, float** k_scale, float** v_scale,
                  int32_t** pos, float** score, int32_t** table, int32_t** meta, int32_t** ref) {
  if (int rc = check_list(p, layer, false, 0, nullptr)) return rc;
  const h2o::PoolView v = layer_view(p, layer);
  if (K) *K = v.K;
  if (V) *V = v.V;
  if (k_scale) *k_scale = v.kscale;
  if (v_scale) *v_scale = v.vscale;
  if (pos) *pos = v.pos;
  if (score) *score = v.score;
  if (table) *table = v.table;
  if (meta) *meta = v.meta;
  if (ref) *ref = v.ref;
  return H2O_OK;
}

int h2o_pool_write(h2o_pool* p, int layer, int n, const int32_t* seqs, const void* K,
                   const void* V, int T, const int32_t* lens, const float* score) {
  if (int rc = check_list(p, layer, false, n, seqs)) return rc;
  if (T < 0 || T > H2O_MAX_T) return fail(H2O_EINVAL, "T out of range");
  if (n == 0) return H2O_OK;
  if (T > 0 && (!K || !V)) return fail(H2O_EINVAL, "null K or V");
  if (!aligned16(K) || !aligned16(V)) return fail(H2O_EINVAL, "K and V must be 16-byte aligned");
  return guarded([&] {
    const h2o::PoolView v = layer_view(p, layer);
    const size_t fresh = static_cast<size_t>(n) * ((T + v.page - 1) / v.page);
    const size_t plan = static_cast<size_t>(n) * h2o::kPlanInts;
    cudaStream_t s = current_stream();
    Scratch mem((fresh + plan) * sizeof(int32_t), s);
    int32_t* m = static_cast<int32_t*>(mem.p);
    return launch_status(h2o::pool_write(v, n, seqs, K, V, T, lens, score, m, m + fresh, s),
                         "pool write launch");
  });
}

int h2o_pool_append(h2o_pool* p, int layer, int n, const int32_t* seqs, const h2o_qkv* x,
                    const h2o_rotary* rotary, int T, const int32_t* lens, const int32_t* parent, void* q_out) {
  if (int rc = check_list(p, layer, false, n, seqs)) return rc;
  h2o::RotateArgs a{};
  if (int rc = rotate_args(x, rotary, n, T, {q_out, nullptr, nullptr}, false, &a)) return rc;
  if (parent && T > H2O_POOL_MAX_NODES) return fail(H2O_EINVAL, "more drafts than H2O_POOL_MAX_NODES");
  if (n == 0) return H2O_OK;
  if (T > 0 && (!x->k.data || !x->v.data)) return fail(H2O_EINVAL, "null k or v");
  if (x->heads != p->v.heads || x->head_dim != p->v.d)
    return fail(H2O_EINVAL, "heads and head_dim must be the pool's");
  return guarded([&] {
    const h2o::PoolView v = layer_view(p, layer);
    const size_t fresh = static_cast<size_t>(n) * ((T + v.page - 1) / v.page);
    const size_t plan = static_cast<size_t>(n) * h2o::kPlanInts;
    cudaStream_t s = current_stream();
    Scratch mem((fresh + plan) * sizeof(int32_t), s);
    int32_t* m = static_cast<int32_t*>(mem.p);
    return launch_status(h2o::pool_append(v, a, seqs, lens, parent, m, m + fresh, s), "pool append launch");
  });
}

int h2o_pool_fork(h2o_pool* p, int layer, int n, const int32_t* src, const int32_t* dst) {
  return fork_or_copy(p, layer, n, src, dst, true);
}

int h2o_pool_copy(h2o_pool* p, int layer, int n, const int32_t* src, const int32_t* dst) {
  return fork_or_copy(p, layer, n, src, dst, false);
}

int h2o_pool_free(h2o_pool* p, int layer, int n, const int32_t* seqs) {
  if (int rc = check_list(p, layer, true, n, seqs)) return rc;
  return guarded([&] {
    return launch_status(h2o::pool_free(layer_view(p, layer < 0 ? 0 : layer),
                                        layer < 0 ? p->layers : 1, n, seqs, current_stream()),
                         "pool free launch");
  });
}

int h2o_pool_compact(h2o_pool* p, int layer, int n, const int32_t* seqs, int h, int r) {
  if (int rc = check_list(p, layer, true, n, seqs)) return rc;
  if (h < 0 || r < 0 || h > H2O_MAX_K || r > H2O_MAX_K || h + r < 1 || h + r > H2O_MAX_K)
    return fail(H2O_EINVAL, "need h >= 0, r >= 0 and 1 <= h + r <= H2O_MAX_K");
  if (n == 0) return H2O_OK;
  return guarded([&] {
    const h2o::PoolView v = layer_view(p, layer < 0 ? 0 : layer);
    // where no sequence can be longer than the budget nothing is kept; the list is checked all the same
    const size_t L = layer < 0 ? p->layers : 1, N = n, k = h + r < v.cap ? h + r : 0;
    const size_t fresh = L * N * ((k + v.page - 1) / v.page), plan = L * N * h2o::kPlanInts;
    const size_t kept = L * N * v.heads * k;
    cudaStream_t s = current_stream();
    Scratch mem((fresh + plan + 2 * kept) * sizeof(int32_t), s);
    int32_t* m = static_cast<int32_t*>(mem.p);
    return launch_status(
        h2o::pool_compact(v, static_cast<int>(L), n, seqs, h, r, m, m + fresh, m + fresh + plan,
                          reinterpret_cast<float*>(m + fresh + plan + kept), s),
        "pool compaction launch");
  });
}

int h2o_pool_attend(h2o_pool* p, int layer, int n, const int32_t* seqs, int prefix, const void* q,
                    int q_heads, void* out, float* lse, int accumulate) {
  if (int rc = check_list(p, layer, false, n, seqs)) return rc;
  if (prefix < -1 || prefix >= p->v.seqs) return fail(H2O_EINVAL, "prefix out of range");
  if (q_heads < 1 || q_heads % p->v.heads || q_heads / p->v.heads > H2O_POOL_MAX_GROUP)
    return fail(H2O_EINVAL,
                "q_heads must be a multiple of the pool's heads, at most H2O_POOL_MAX_GROUP times");
  if (n == 0) return H2O_OK;
  if (!q || !out) return fail(H2O_EINVAL, "null q or out");
  if (!aligned16(q) || !aligned16(out)) return fail(H2O_EINVAL, "q and out must be 16-byte aligned");
  const size_t bytes = static_cast<size_t>(n) * q_heads * p->v.d * 2;
  const size_t lse_bytes = lse ? static_cast<size_t>(n) * q_heads * sizeof(float) : 0;
  if (overlap(q, bytes, out, bytes) || overlap(lse, lse_bytes, q, bytes) ||
      overlap(lse, lse_bytes, out, bytes))
    return fail(H2O_EINVAL, "q, out and lse must not overlap");
  return guarded([&] {
    h2o::AttendArgs a{};
    a.v = layer_view(p, layer);
    a.seqs = seqs;
    a.n = n;
    a.prefix = prefix;
    a.group = q_heads / p->v.heads;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.accumulate = accumulate != 0;
    a.kmap = &p->maps[2 * layer];
    a.vmap = &p->maps[2 * layer + 1];
    cudaStream_t s = current_stream();
    // The scratch grows with the batch and, for the scores, with the longest sequence that the
    // pool can hold, whatever the lengths are. Where there is not that much memory the batch
    // goes in parts, one after the other through the same scratch, which is there before the first.
    for (int part = n;; part = (part + 1) / 2) {
      auto sized = [&](int entries) {
        h2o::AttendArgs x = a;
        x.n = entries;
        return h2o::pool_attend_scratch(x);
      };
      // (a last part of few entries can need more than a full one)
      const size_t need = std::max(sized(part), n % part ? sized(n % part) : 0);
      std::unique_ptr<Scratch> mem;
      try {
        mem = std::make_unique<Scratch>(need, s);
      } catch (const std::exception&) {
        if (part == 1) throw;
        continue;
      }
      for (int at = 0; at < n; at += part) {
        const size_t row = static_cast<size_t>(at) * q_heads;
        a.before = at;
        a.n = std::min(part, n - at);
        a.seqs = seqs + at;
        a.q = static_cast<const uint8_t*>(q) + row * p->v.d * 2;
        a.out = static_cast<uint8_t*>(out) + row * p->v.d * 2;
        a.lse = lse ? lse + row : nullptr;
        cudaError_t e = h2o::pool_attend(a, mem->p, s);
        if (e != cudaSuccess) return cuda_fail(e, "pool attention launch");
      }
      return static_cast<int>(H2O_OK);
    }
  });
}

int h2o_pool_attend_tree(h2o_pool* p, int layer, int n, const int32_t* seqs, int prefix, const void* q,
                         int q_heads, int T, const int32_t* lens, const int32_t* parent, void* out, float* lse) {
  if (int rc = check_list(p, layer, false, n, seqs)) return rc;
  if (prefix < -1 || prefix >= p->v.seqs) return fail(H2O_EINVAL, "prefix out of range");
  if (q_heads < 1 || q_heads % p->v.heads || q_heads / p->v.heads > H2O_POOL_MAX_GROUP)
    return fail(H2O_EINVAL,
                "q_heads must be a multiple of the pool's heads, at most H2O_POOL_MAX_GROUP times");
  if (T < 0 || T > H2O_POOL_MAX_NODES) return fail(H2O_EINVAL, "T must be in [0, H2O_POOL_MAX_NODES]");
  if (n == 0 || T == 0) return H2O_OK;
  if (!q || !out) return fail(H2O_EINVAL, "null q or out");
  if (!aligned16(q) || !aligned16(out)) return fail(H2O_EINVAL, "q and out must be 16-byte aligned");
  const size_t rows = static_cast<size_t>(n) * T * q_heads, bytes = rows * p->v.d * 2;
  if (rows >> 31) return fail(H2O_EINVAL, "2^31 rows or more");
  const size_t lse_bytes = lse ? rows * sizeof(float) : 0;
  if (overlap(q, bytes, out, bytes) || overlap(lse, lse_bytes, q, bytes) || overlap(lse, lse_bytes, out, bytes))
    return fail(H2O_EINVAL, "q, out and lse must not overlap");
  return guarded([&] {
    h2o::AttendArgs a{};
    a.v = layer_view(p, layer);
    a.seqs = seqs;
    a.n = n * T;
    a.prefix = prefix;
    a.group = q_heads / p->v.heads;
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.kmap = &p->maps[2 * layer];
    a.vmap = &p->maps[2 * layer + 1];
    const h2o::TreeArgs t{n, T, lens, parent};
    cudaStream_t s = current_stream();
    Scratch mem(h2o::pool_tree_scratch(a, t), s);
    return launch_status(h2o::pool_tree(a, t, mem.p, s), "tree attention launch");
  });
}

int h2o_pool_accept(h2o_pool* p, int layer, int n, const int32_t* seqs, int T, const int32_t* lens,
                    const int32_t* path, int P, const void* q, int q_heads, const float* lse, int prefix) {
  if (int rc = check_list(p, layer, !q, n, seqs)) return rc;
  if (T < 0 || T > H2O_POOL_MAX_NODES) return fail(H2O_EINVAL, "T must be in [0, H2O_POOL_MAX_NODES]");
  if (P < 0 || P > H2O_POOL_MAX_NODES) return fail(H2O_EINVAL, "P must be in [0, H2O_POOL_MAX_NODES]");
  if (n > 0 && P > 0 && !path) return fail(H2O_EINVAL, "null path");
  if (q) {
    if (!lse) return fail(H2O_EINVAL, "q without lse");
    if (prefix < -1 || prefix >= p->v.seqs) return fail(H2O_EINVAL, "prefix out of range");
    if (q_heads < 1 || q_heads % p->v.heads || q_heads / p->v.heads > H2O_POOL_MAX_GROUP)
      return fail(H2O_EINVAL,
                  "q_heads must be a multiple of the pool's heads, at most H2O_POOL_MAX_GROUP times");
    if (!aligned16(q)) return fail(H2O_EINVAL, "q must be 16-byte aligned");
  } else if (lse) {
    return fail(H2O_EINVAL, "lse without q");
  }
  if (n == 0) return H2O_OK;
  return guarded([&] {
    const h2o::PoolView v = layer_view(p, layer < 0 ? 0 : layer);
    const size_t L = layer < 0 ? p->layers : 1, N = n;
    const size_t plan = L * N * h2o::kAcceptInts, sums = q ? N + 1 : 0, kept = q ? N * P : 0;
    cudaStream_t s = current_stream();
    Scratch mem((plan + 2 * sums + kept) * sizeof(int32_t), s);
    int32_t* m = static_cast<int32_t*>(mem.p);
    int32_t *rows = q ? m + plan : nullptr, *tiles = q ? rows + sums : nullptr, *list = q ? tiles + sums : nullptr;
    cudaError_t e = h2o::pool_accept(v, static_cast<int>(L), n, seqs, T, lens, path, P, q ? prefix : -1, m, rows,
                                     tiles, list, s);
    if (e == cudaSuccess && q && T > 0 && P > 0) {
      const h2o::AcceptArgs a{v, seqs, n, prefix, q_heads / v.heads, q, lse, m, rows, tiles, list};
      e = h2o::pool_accept_scores(a, s);
    }
    return launch_status(e, "pool accept launch");
  });
}

int h2o_pool_sync_check(h2o_pool* p) {
  if (int rc = check_pool(p)) return rc;
  return guarded([&] { return check_error_word(p->v.err, current_stream()); });
}

}  // extern "C"
