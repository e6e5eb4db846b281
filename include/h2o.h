/*
 * h2o.h - C ABI of the GB300 (sm_103a) H2O heavy-hitter KV-cache library.
 *
 * Sources (page title and section):
 *   [H2O] "H2O: Heavy-Hitter Oracle for Efficient Generative Inference of Large
 *         Language Models", section-by-section summary page of arXiv 2306.14048v3.
 *
 * The policy keeps, for every (layer, batch row, head) "row", at most
 * k = h + r cached tokens: h heavy hitters and the r most recent tokens
 * ([H2O] A, System Details). A token's accumulated score is the running sum of
 * the softmax probabilities it has received ([H2O] 1, 3.2). At most one token is
 * evicted per decoding step and the cache never exceeds k ([H2O] TL;DR, 2).
 *
 * Conventions shared by every entry point
 *   - Return value: H2O_OK (0) on success, a negative H2O_E* code on failure.
 *     h2o_last_error() then returns a message for the calling thread. No entry
 *     point traps or aborts; device kernels never trap. Bounded device waits
 *     that give up set a device error word that h2o_sync_check() reports.
 *   - Device pointers are CUDA device addresses on the current device; host
 *     pointers are ordinary CPU memory. Every buffer passed in stays owned by
 *     the caller and is only accessed by work the call enqueues. A context
 *     belongs to the device that was current when it was created: an entry
 *     point given a context returns H2O_EINVAL while another device is current.
 *   - All device work is enqueued, asynchronously, on the calling thread's
 *     current PyTorch CUDA stream (c10::cuda::getCurrentCUDAStream()). The
 *     caller must have initialised PyTorch's CUDA state on that device
 *     (torch.cuda.init() or any CUDA tensor). Only h2o_cache_positions,
 *     h2o_last_evicted and h2o_sync_check synchronise with the host.
 *   - The library owns the cache. It allocates it from PyTorch's CUDA caching
 *     allocator and frees it in h2o_destroy. PyTorch serves for nothing else.
 *   - Prompt tensors Q, K, V and prefill outputs `out` are moved by TMA and
 *     must be 16-byte aligned (any CUDA allocation is); otherwise H2O_EINVAL.
 *   - Layouts: Q, K, V of a prompt are bf16, contiguous [batch, heads, T, d];
 *     decode inputs q, k_new, v_new are bf16, contiguous [batch, heads, d];
 *     outputs are fp32 in the same layouts. head_dim d is 64 or 128. Logits
 *     are scaled by 1/sqrt(d).
 *   - Position t counts tokens of a row from 0: prompt tokens are 0 .. T-1 and
 *     decode step s processes position T + s.
 */
#ifndef H2O_H
#define H2O_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define H2O_OK 0
#define H2O_EINVAL (-1)  /* bad argument (null pointer, size out of range, layer out of range) */
#define H2O_ESTATE (-2)  /* call not valid in the current state (decode before prefill, or a
                            second prefill of a layer without h2o_reset) */
#define H2O_ENOMEM (-3)  /* device allocation failed */
#define H2O_ECUDA (-4)   /* a CUDA runtime call or kernel launch failed */
#define H2O_EDEVICE (-5) /* a kernel reported an error through the device error word */

#define H2O_MAX_T (1 << 20)  /* longest prompt accepted by h2o_prefill */
#define H2O_MAX_K 32768      /* largest budget h + r accepted by h2o_create */

#define H2O_KV_BF16 0  /* cache keys and values stored as bf16 (h2o_create) */
#define H2O_KV_FP8 1   /* cache keys and values stored as E4M3 codes with per-token scales */
#define H2O_LAYOUT_RING 0x100 /* OR into kv_format: heavy slots, then the window as a circular queue */

typedef struct h2o_ctx h2o_ctx; /* opaque; created by h2o_create, freed by h2o_destroy */

/*
 * h2o_create - allocate the cache of a model: `layers` layers of batch x heads
 * rows, each with a budget of h heavy-hitter plus r recent tokens ([H2O] A,
 * System Details: preallocated cache with a heavy-hitter and a recent region).
 *
 * Per layer the cache holds, for rows = batch * heads and k = h + r slots:
 *   K, V   bf16  [rows][k][d]   cached keys / values, slot-indexed (E4M3
 *                               codes, uint8, for an h2o_create_ex FP8 cache)
 *   score  fp32  [rows][k]      accumulated attention score of each slot
 *   pos    int32 [rows][k]      token position held by each slot (-1 = empty)
 *   meta   int32 [rows][4]      {filled slots, next position t, last evicted position (-1 none), 0}
 * Slots [0, filled) are occupied; slot order carries no meaning.
 *
 * Arguments: layers >= 1, batch >= 1, heads >= 1, head_dim in {64, 128},
 * h >= 0, r >= 0, 1 <= h + r <= H2O_MAX_K. *out receives the new context.
 * Errors: H2O_EINVAL, H2O_ENOMEM, H2O_ECUDA. On error *out is set to NULL.
 */
int h2o_create(int layers, int batch, int heads, int head_dim, int h, int r, h2o_ctx** out);

/*
 * h2o_create_ex - h2o_create with a choice of cache storage. The pages report
 * that H2O combines with quantisation of the KV cache and that the combination
 * beats either alone ([H2O] 5, Empirical Evaluation), without fixing a scheme.
 * kv_format H2O_KV_FP8 stores every cached token's key and value vectors as
 * E4M3 codes (OCP 8-bit floating point: 1 sign, 4 exponent bits with bias 7, 3
 * mantissa bits, largest finite value 448) with one fp32 scale per vector:
 * scale = amax / 448 and code = E4M3(x * (448 / amax)), round to nearest even,
 * saturated; a zero vector has scale 0. The arithmetic is fp32 with one
 * rounding per operation. Prefill attention still runs on the full-precision
 * prompt and the kept tokens are quantised as they enter the cache; a decode
 * step quantises the new token first and attends to the stored (dequantised)
 * values of every cached token, the new one included. Per layer the cache then
 * holds K, V as uint8 [rows][k][d] and two fp32 [rows][k] scale arrays
 * (h2o_cache_scales), 2d + 8 bytes per slot instead of 4d.
 * kv_format H2O_KV_BF16 is h2o_create. Other arguments and errors as for
 * h2o_create; an unknown kv_format gives H2O_EINVAL.
 *
 * kv_format H2O_KV_BF16 | H2O_LAYOUT_RING (needs r >= 1) lays each row's
 * slots out as the pages' implementation does ([H2O] A, System Details: a
 * heavy-hitter region and the recent tokens in a circular queue): heavy slots
 * [0, h) in use from slot 0, and the token at recent position p in slot
 * h + p mod r. The decode step then reads no position of a recent slot (they
 * follow from t); its candidates are the heavy slots and the token leaving
 * the window, which moves into the heavy slot it displaces. Results are those
 * of the default slot-indexed layout (outputs, evictions, retained sets);
 * only the slot order differs. h2o_decode_steps takes one launch per step.
 */
int h2o_create_ex(int layers, int batch, int heads, int head_dim, int h, int r, int kv_format,
                  h2o_ctx** out);

/* h2o_destroy - free the cache and the context. Waits for the context's
 * stream work to finish first. NULL is accepted. */
void h2o_destroy(h2o_ctx* ctx);

/*
 * h2o_prefill - prompt pass of one layer ([H2O] A, Pseudocode: a prompt of at
 * least 2K tokens keeps K heavy hitters and K recent tokens).
 *
 * For every row: causal softmax attention of the T prompt queries over the
 * prompt keys, written to out; the accumulated score of prompt token j is the
 * column sum sum_{i >= j} P_ij of the causal probability matrix ([H2O] 3.2);
 * the cache then holds the r most recent tokens T-r .. T-1 plus the h other
 * tokens with the largest (score, position) keys, or every token if T <= h + r.
 * Ties in score keep the later position. Retained tokens keep their column
 * sums as accumulated scores.
 *
 * State: a layer takes one prompt ([H2O] A, Pseudocode: the prompt's heavy
 * hitters are selected once, then generation proceeds step by step). The
 * layer must be empty, as h2o_create or h2o_reset leaves it; a second prefill
 * without h2o_reset returns H2O_ESTATE and changes nothing. After a prefill
 * that fails the layer still counts as empty: decode returns H2O_ESTATE and
 * the next prefill is accepted.
 *
 * Q, K, V: device bf16 [batch, heads, T, d]; out: device fp32 [batch, heads, T, d].
 * 0 <= T <= H2O_MAX_T; with T = 0 the pointers may be NULL and the layer is
 * reset to an empty cache. Scratch (per-row log-sum-exp and column sums,
 * 8 bytes per prompt token) comes from PyTorch's caching allocator on the
 * current stream. Errors: H2O_EINVAL, H2O_ESTATE (layer not empty), H2O_ENOMEM,
 * H2O_ECUDA.
 */
int h2o_prefill(h2o_ctx* ctx, int layer, const void* Q, const void* K, const void* V, int T,
                float* out);

/*
 * h2o_reset - return one layer (layer >= 0) or every layer (layer = -1) to the
 * empty state h2o_create leaves: no token cached (positions -1, scores 0, fill
 * count and next position 0), ready for a new prompt (h2o_prefill). Enqueues
 * one small kernel per layer on the current stream; allocates nothing.
 * Errors: H2O_EINVAL (null context, layer out of range), H2O_ECUDA.
 */
int h2o_reset(h2o_ctx* ctx, int layer);

/*
 * h2o_prefill_ragged - h2o_prefill of a batch whose prompts differ in length
 * ([H2O] 5, Empirical Evaluation, Throughput and Latency: the gains come from
 * serving larger batches; entries of a batch are independent sequences, and
 * their prompts need not be equally long).
 *
 * Batch entry b holds a prompt of T_b = lens[b] tokens, stored right-padded
 * to T_max: Q, K, V device bf16 [batch, heads, T_max, d] with token t of entry
 * b at index t for t < T_b. Each row is processed exactly as h2o_prefill
 * processes a prompt of T_b tokens (attention, column sums, the r most recent
 * tokens T_b - r .. T_b - 1 plus the top-h others, or all T_b tokens when
 * T_b <= h + r), and its first decode step then processes position T_b.
 *
 * lens: device int32 [batch], 0 <= lens[b] <= T_max, read on the device (the
 * call can be captured in a CUDA graph with lengths written later). A length
 * outside that range is clamped into it and sets bit 4 of the device error
 * word (h2o_sync_check reports H2O_EDEVICE). The padding tokens t >= T_b of
 * Q, K and V must hold finite values (zeros, say): padded keys and values
 * enter the tensor-core products with probability 0, and 0 times a non-finite
 * value is not 0. out: device fp32 [batch, heads, T_max, d]; rows t >= T_b
 * hold no result (the call may write them). Scratch as for h2o_prefill, sized
 * by T_max. With T_max = 0 the pointers may be NULL and every row is reset to
 * an empty cache. The layer must be empty, as for h2o_prefill. Errors:
 * H2O_EINVAL (also for lens NULL with T_max > 0), H2O_ESTATE, H2O_ENOMEM,
 * H2O_ECUDA.
 */
int h2o_prefill_ragged(h2o_ctx* ctx, int layer, const void* Q, const void* K, const void* V,
                       int T_max, const int32_t* lens, float* out);

/*
 * h2o_decode_step - one generation step of one layer ([H2O] 4.1 and 2).
 *
 * For every row, with t its next position: append the new token (q, k_new,
 * v_new); attend over the cached tokens plus the new one, writing
 * out = sum_j p_j v_j with p = softmax(K q / sqrt(d)); add p_j to every cached
 * token's accumulated score and give the new token score p_t; if the row now
 * holds more than k tokens, evict the token with the smallest (score, position)
 * among those at positions <= t - r (the r most recent, t included, are never
 * evicted; with r = 0 the new token competes and may be dropped at once); the
 * new token's K/V, position and score go into the freed slot, or into the next
 * empty slot while the cache is not full.
 *
 * q, k_new, v_new: device bf16 [batch, heads, d]; out: device fp32 [batch, heads, d].
 * Allocates nothing and never synchronises. The step position and fill count
 * live in device memory and are advanced by the kernel, so the call can be
 * captured in a CUDA graph and replayed. Errors: H2O_EINVAL, H2O_ESTATE (layer
 * never prefilled), H2O_ECUDA.
 *
 * The kernel checks each row's state before it touches the row: a fill count
 * outside [0, k] or above the next position t, or an occupied slot whose
 * position is outside [0, t) (a state installed through h2o_cache_view that
 * no call of this library produces), sets bit 2 (bad state) of the device
 * error word, and a row with inconsistent counts is left unchanged.
 * h2o_sync_check then reports H2O_EDEVICE.
 */
int h2o_decode_step(h2o_ctx* ctx, int layer, const void* q, const void* k_new, const void* v_new,
                    float* out);

/*
 * h2o_decode_steps - `steps` consecutive h2o_decode_step calls of one layer
 * whose inputs are all known in advance ([H2O] 4.1: the policy is the same
 * greedy step repeated; 5, Ablation and Extended Evaluations: streaming over
 * long inputs), e.g. a teacher-forced pass over a known continuation, one
 * layer after the other. Results equal those of the single steps.
 *
 * q, k_new, v_new: device bf16 [steps, batch, heads, d]; out: device fp32
 * [steps, batch, heads, d]; evicted: device int32 [steps, batch * heads], the
 * position evicted by each row at each step (-1: none, the new token's own
 * position when it is dropped), or NULL. With h + r <= 8192 all steps run in
 * one launch, one CTA per row looping over its steps (no per-step launch and
 * drain); larger budgets, and rows of 1024 slots or more when there are fewer
 * rows than SMs (where splitting rows over several CTAs moves the bytes
 * faster), take one launch per step. steps >= 0 (0: nothing is
 * done). Allocates nothing and never synchronises; capturable in a CUDA
 * graph. Errors: H2O_EINVAL, H2O_ESTATE (layer never prefilled), H2O_ECUDA.
 */
int h2o_decode_steps(h2o_ctx* ctx, int layer, int steps, const void* q, const void* k_new,
                     const void* v_new, float* out, int32_t* evicted);

/*
 * h2o_prefill_attention - the attention part of prefill, without touching any
 * cache: causal attention of `rows` independent rows of T tokens, the output
 * and every token's column-sum score.
 *
 * Q, K, V: device bf16 [rows, T, d]; out: device fp32 [rows, T, d];
 * score: device fp32 [rows, T]. Scratch (per-row log-sum-exp, 4 bytes per
 * token) comes from PyTorch's caching allocator on the current stream.
 * A bounded device wait that gives up is reported through the library's own
 * error word (h2o_attention_sync_check), since no context is involved.
 * Errors: H2O_EINVAL, H2O_ENOMEM, H2O_ECUDA.
 */
int h2o_prefill_attention(const void* Q, const void* K, const void* V, int rows, int T,
                          int head_dim, float* out, float* score);

/*
 * h2o_prefill_attention_noalloc - the same computation as h2o_prefill_attention
 * (outputs and column-sum scores of `rows` cache-free rows), for callers that
 * must not allocate device memory during the call. The pages have no
 * counterpart to this entry point; it exists for the caller, not the policy.
 *
 * Who needs it: callers for which a device allocation during the call is not
 * an option. A serving process may reserve its device memory once at start-up
 * and forbid allocation on the request path, because cudaMalloc can block
 * until the device is idle and stall every stream. A process whose memory is
 * pre-reserved by another framework's arena (one that grabs most of the GPU up
 * front) has little free memory left, so an extra allocation can fail there.
 * Such callers cannot use h2o_prefill_attention, whose per-row log-sum-exp
 * scratch comes from PyTorch's caching allocator.
 *
 * Instead the scratch is a fixed device array inside the library
 * (H2O_NOALLOC_MAX_LSE floats, 4 MiB, held by every GPU that loads the
 * library until the process exits). This call allocates nothing, uses no
 * PyTorch state and enqueues its kernels on `stream` (a cudaStream_t; NULL is
 * the legacy default stream). The first call on a device looks up the array's
 * device address (cudaGetSymbolAddress) with that device current; make that
 * first call before any stream capture. All calls share the one array, so
 * calls whose work overlaps on the GPU (different streams, or different
 * threads without ordering between them) race on it; calls on one stream are
 * ordered and safe. Nothing in the array needs to start at zero: every entry a
 * call reads was written earlier by the same call.
 *
 * Where the array lives: CUDA loads a library's device code, and with it this
 * array, into a device on first use (lazy module loading is the default), so
 * the first call on each device may itself need 4 MiB of free device memory.
 * Make one small call on each device at start-up, before an arena reserves the
 * rest of the memory (and before any stream capture). The looked-up address
 * belongs to the device's context: after cudaDeviceReset on that device, call
 * h2o_forget_device_state() before the next call, which then looks it up
 * again.
 *
 * Errors inside the kernels: a bounded device wait that gives up sets the
 * library's error word, which h2o_attention_sync_check(stream) reports (the
 * word is also a fixed device variable, not an allocation).
 *
 * Q, K, V: device bf16 [rows, T, d]; out: device fp32 [rows, T, d];
 * score: device fp32 [rows, T]. Limit: rows * (T rounded up to a multiple of
 * 128) <= H2O_NOALLOC_MAX_LSE; larger calls are rejected with H2O_EINVAL and
 * a message. Errors: H2O_EINVAL, H2O_ECUDA.
 */
#define H2O_NOALLOC_MAX_LSE (1 << 20)
int h2o_prefill_attention_noalloc(const void* Q, const void* K, const void* V, int rows, int T,
                                  int head_dim, float* out, float* score, void* stream);

/*
 * h2o_attention_sync_check - synchronise `stream` (a cudaStream_t; NULL is the
 * legacy default stream) and report, then clear, the library-level device
 * error word of the current device that the cache-free entry points
 * (h2o_prefill_attention, h2o_prefill_attention_noalloc) write: bit 1 when
 * one of their bounded waits gave up (their outputs are then incomplete).
 * Allocates nothing. The word is shared by every such call on the device.
 * Errors: H2O_ECUDA, H2O_EDEVICE.
 */
int h2o_attention_sync_check(void* stream);

/*
 * h2o_attention_test_wait_limit - the failure path of the cache-free entry
 * points on demand: enqueues on `stream` one kernel whose bounded wait is
 * never satisfied; after the wait limit (2 s) it sets bit 1 of the
 * library-level error word and returns. The next h2o_attention_sync_check
 * reports H2O_EDEVICE. Errors: H2O_ECUDA.
 */
int h2o_attention_test_wait_limit(void* stream);

/*
 * h2o_forget_device_state - drop the per-device state the library caches (the
 * device addresses of its fixed arrays and its kernels' shared-memory
 * opt-ins), so that the next call on each device sets it up again. Needed
 * only after cudaDeviceReset (which discards a device's context, and with it
 * the library's loaded code and arrays); call it with no work of the library
 * in flight. Contexts made by h2o_create do not survive a device reset.
 */
void h2o_forget_device_state(void);

/*
 * h2o_test_fail_allocations - fault injection on the host: the next n device
 * allocations the library makes (a cache in h2o_create, prefill scratch) fail
 * as an exhausted allocator would, and the calls return H2O_ENOMEM with the
 * state unchanged (no context is created; a layer whose prefill failed stays
 * empty). n = 0 ends it. No GPU work is involved. Errors: H2O_EINVAL (n < 0).
 */
int h2o_test_fail_allocations(int n);

/*
 * h2o_cache_positions - copy the positions held by every slot of one layer to
 * host memory: host_pos int32 [batch * heads * k], row-major by (row, slot),
 * -1 for empty slots. Synchronises the current stream.
 * Errors: H2O_EINVAL, H2O_ECUDA, H2O_EDEVICE.
 */
int h2o_cache_positions(h2o_ctx* ctx, int layer, int32_t* host_pos);

/*
 * h2o_last_evicted - copy, per row, the position evicted by the layer's last
 * decode step (-1 when the step evicted nothing): host_pos int32
 * [batch * heads]. Synchronises the current stream.
 * Errors: H2O_EINVAL, H2O_ECUDA, H2O_EDEVICE.
 */
int h2o_last_evicted(h2o_ctx* ctx, int layer, int32_t* host_pos);

/*
 * h2o_cache_view - device addresses of one layer's cache arrays (layouts as in
 * h2o_create). The library keeps ownership; the addresses stay valid until
 * h2o_destroy. A caller may write through them (between calls, on the same
 * stream) to install a cache state; the fill count in meta must then match the
 * occupied slots, which are slots 0 .. filled-1 of the slot-indexed layout, or
 * for H2O_LAYOUT_RING the tokens older than the window from slot 0 and window
 * position p in slot h + p mod r. Any output pointer may be NULL.
 * Errors: H2O_EINVAL.
 */
int h2o_cache_view(h2o_ctx* ctx, int layer, void** K, void** V, float** score, int32_t** pos,
                   int32_t** meta);

/*
 * h2o_cache_scales - device addresses of one layer's per-slot scales of an
 * H2O_KV_FP8 cache: k_scale, v_scale fp32 [rows][k] (a slot's stored key is
 * E4M3(code) * k_scale). Same ownership and lifetime as h2o_cache_view; any
 * output pointer may be NULL. Errors: H2O_EINVAL (also for a bf16 cache).
 */
int h2o_cache_scales(h2o_ctx* ctx, int layer, float** k_scale, float** v_scale);

/* h2o_cache_dims - k (slots per row) and rows (batch * heads) per layer. */
int h2o_cache_dims(h2o_ctx* ctx, int* k, int* rows);

/*
 * h2o_test_wait_limit - the failure path on demand: enqueues one kernel whose
 * bounded mbarrier wait is never satisfied (nothing arrives on the barrier).
 * Like any kernel of the library whose producer never delivers, it gives up
 * after the wait limit (2 s), sets bit 1 (wait timeout) of the context's
 * device error word and returns; no kernel traps. The next h2o_sync_check
 * reports H2O_EDEVICE and clears the word, and the context stays usable.
 * Errors: H2O_EINVAL, H2O_ECUDA.
 */
int h2o_test_wait_limit(h2o_ctx* ctx);

/*
 * h2o_sync_check - synchronise the current stream and report, then clear, the
 * context's device error word. Errors: H2O_ECUDA, H2O_EDEVICE.
 */
int h2o_sync_check(h2o_ctx* ctx);

/*
 * ---- Rotary positions ------------------------------------------------------
 *
 * Models that rotate queries and keys by their positions call h2o_rotate_qkv on a
 * projection's output before h2o_prefill, h2o_prefill_attention, h2o_pool_write or
 * h2o_decode_step, whose inputs it lays out, and h2o_pool_append in the place of
 * h2o_pool_write where the pool knows the positions. The pages describe the policy
 * for vectors as they are; these entry points make them.
 *
 * The first `dim` channels of a head are dim / 2 pairs: channels (i, i + dim / 2)
 * with H2O_ROTARY_HALF, (2 i, 2 i + 1) with H2O_ROTARY_INTERLEAVED. At position p
 * pair i becomes factor * (x cos a - y sin a, x sin a + y cos a) with a = p f_i; other
 * channels stay. Angles are exact for every 32-bit p and the f_i that are given, as fp64,
 * up to the rounding of f_i to 2^-64 of a turn and of a to fp32 (2 pi 2^-26).
 */
#define H2O_ROTARY_HALF 0
#define H2O_ROTARY_INTERLEAVED 1
#define H2O_ROTARY_MAX_PAIRS 64
#define H2O_ROTARY_MAX_HEADS 32768 /* most heads of q, k or v in one call */

/* A plain value without resources: made by h2o_rotary_init, read during a call only. */
typedef struct h2o_rotary {
  int32_t dim;    /* rotated channels: a multiple of 16 in [0, 128], at most head_dim */
  int32_t layout; /* H2O_ROTARY_* */
  float factor;   /* of cosines and sines */
  uint32_t reserved;
  uint64_t turns[H2O_ROTARY_MAX_PAIRS]; /* f_i / (2 pi) without whole turns, times 2^64 */
} h2o_rotary;

#define H2O_ROTARY_PLAIN 0  /* f_i = base^(-2 i / dim) */
#define H2O_ROTARY_LINEAR 1 /* f_i / factor: positions interpolated */
#define H2O_ROTARY_NTK 2    /* base * factor^(dim / (dim - 2)) for the base */
#define H2O_ROTARY_PARTS 3  /* g f_i + (1 - g) f_i / factor, g = clamp((original f_i / (2 pi) - low) /
                               (high - low), 0, 1): pairs that turn more than `high` times in the
                               `original` context stay, those that turn less than `low` times are
                               interpolated. Pass the attention factor that goes with it, such as
                               0.1 ln(factor) + 1, to h2o_rotary_init. */

/*
 * h2o_rotary_frequencies - dim / 2 frequencies in radians a position, host memory.
 * dim a multiple of 16 in [16, 128]; what a scaling does not name is ignored. (Powers
 * and products in fp64: relative errors of some 2^-49, which times p are the angle's.)
 * h2o_rotary_init - the rotation by given frequencies (host memory; any values of
 * magnitude up to 2^53; NULL with dim = 0, which rotates nothing). No GPU work. Errors: H2O_EINVAL.
 */
int h2o_rotary_frequencies(int dim, double base, int scaling, double factor, double original,
                           double low, double high, double* frequencies);
int h2o_rotary_init(h2o_rotary* out, int dim, int layout, const double* frequencies, double factor);

/* bf16 [batch][T][heads][d], 16-byte aligned: strides in elements, multiples of 8 in [0, 2^30 d] that
 * reach no further than 2^60 elements (of sizes above 1); channels are contiguous. data NULL: not there. */
typedef struct h2o_heads {
  const void* data;
  int64_t batch, token, head;
} h2o_heads;

/* A projection's output. q_norm, k_norm: device fp32 [head_dim], 16-byte aligned, weights w of the norm x <-
 * x w / sqrt(mean(x^2) + eps) of every head before its rotation (sums in fp32: heads whose squares sum up
 * beyond it become 0), or NULL: no norm. */
typedef struct h2o_qkv {
  h2o_heads q, k, v;
  int32_t q_heads, heads, head_dim; /* heads: of k and v */
  float eps;
  const float *q_norm, *k_norm;
} h2o_qkv;

/*
 * h2o_rotate_qkv - norms and rotates queries and keys, and lays out queries, keys
 * and values: q_out bf16 [batch][q_heads][T][d], k_out and v_out [batch][heads][T][d],
 * contiguous and 16-byte aligned, NULL for what is not there. Each result is rounded
 * once from fp32; values are copied. positions: device int32 [batch][T], NULL: 0 ..
 * T - 1; rotary NULL: nothing is rotated. Outputs must not lie between the first and
 * the last element of an input, nor on each other. 0 <= T <= H2O_MAX_T, batch * T
 * < 2^31, head_dim 64 or 128. Allocates nothing. Errors: H2O_EINVAL, H2O_ECUDA.
 */
int h2o_rotate_qkv(const h2o_qkv* x, const h2o_rotary* rotary, int batch, int T,
                   const int32_t* positions, void* q_out, void* k_out, void* v_out);

/*
 * ---- Paged cache -----------------------------------------------------------
 *
 * A pool holds sequences of different lengths in pages that sequences can
 * share, next to the fixed slot cache of h2o_create: for batches whose members
 * come and go, are forked (samples, beams) or begin with the same long prefix.
 * The policy is applied by h2o_pool_compact, at the moments the caller picks.
 *
 * Per layer, with N pages of `page` tokens, S sequences of at most W pages
 * (C = W * page tokens) and H key/value heads, a pool holds
 *   K, V   bf16  [N][H][page][d]  stored keys / values (E4M3 codes, uint8, in
 *                                 an H2O_KV_FP8 pool, quantised as h2o_create_ex
 *                                 describes but for the two cases below, with
 *                                 fp32 [N][H][page] scales each)
 *   pos    int32 [N][H][page]     position of the token a slot holds
 *   score  fp32  [S][H][C]        accumulated score of each slot of a sequence
 *   table  int32 [S][W]           pages of a sequence in order, -1 behind the last
 *   meta   int32 [S][2]           {tokens held, next position}
 *   ref    int32 [N]              sequences that hold a page; 0 = free
 * Token i of a sequence is in slot i mod page of page table[i / page]. Heads
 * keep different tokens after a compaction, in ascending order of position.
 * Scores belong to the sequence, keys, values and positions to the page. Whole
 * pages may be shared and are never written again; the partial last page of a
 * sequence is its own. Slots behind a sequence's last token hold no result.
 * An H2O_KV_FP8 pool stores a vector of magnitude up to 2^-119, whose 448 / amax
 * fp32 does not hold, as a zero vector, and one with a NaN or an infinity as zero
 * codes with a NaN for their scale: it reads as NaN in every channel.
 *
 * Lists. `seqs`, `src` and `dst` are device int32 [n], read on the device, n <=
 * H2O_POOL_MAX_LIST; entries of -1 are skipped (a padded batch). An index
 * outside the pool, or one named earlier in the list, sets bit 16 (bad list) of
 * the pool's error word and its entry is skipped; only `src` may name a
 * sequence twice. The operators that need pages take the free pages of lowest
 * index, for the entries in order of the list; when they run out, that entry
 * and all after it are refused, unchanged, with bit 8 (no page). A state
 * that no call leaves (a length or a page out of range, installed through
 * h2o_pool_view) sets bit 2 and is not followed. h2o_pool_sync_check reports
 * the bits as H2O_EDEVICE.
 *
 * layer: >= 0, or -1 for all layers at once where that is said. Calls are
 * enqueued on the current stream, never synchronise, and can be captured in a
 * CUDA graph; scratch comes from PyTorch's caching allocator. Calls on one
 * layer of a pool change its state, so they have to be ordered (one stream, or
 * events); different layers and pools are independent but for the error word.
 */
typedef struct h2o_pool h2o_pool;

#define H2O_POOL_MAX_LIST 1024  /* longest sequence list of one call */
#define H2O_POOL_MAX_HEADS 1024 /* most key/value heads of a pool */
#define H2O_POOL_MAX_NODES 64   /* most drafted tokens of a sequence in one call */
#define H2O_POOL_MAX_GROUP 32   /* most query heads per key/value head (h2o_pool_attend) */

/*
 * h2o_pool_create - allocate a pool: every page free, every sequence empty.
 * layers >= 1, pages >= 1, page_size in {16, 32, 64, 128}, head_dim in {64,
 * 128}, 1 <= heads <= H2O_POOL_MAX_HEADS, 1 <= sequences <= 2^20, max_pages >=
 * 1 pages per sequence with max_pages * page_size <= H2O_MAX_T, and pages *
 * heads * page_size < 2^31. kv_format H2O_KV_BF16 or H2O_KV_FP8.
 * Errors: H2O_EINVAL, H2O_ENOMEM, H2O_ECUDA; *out is then NULL.
 */
int h2o_pool_create(int layers, int pages, int page_size, int heads, int head_dim, int sequences,
                    int max_pages, int kv_format, h2o_pool** out);

/* h2o_pool_destroy - wait for the device's work, then free the pool. NULL is
 * accepted. While the current stream is captured nothing is waited for: the
 * pool's work on other streams must then have finished. */
void h2o_pool_destroy(h2o_pool* pool);

/* h2o_pool_view - device addresses of one layer's arrays; the layers of an
 * array lie one after the other. Same ownership and rules as h2o_cache_view; a
 * bf16 pool has no scales (NULL). Any output pointer may be NULL.
 * Errors: H2O_EINVAL. */
int h2o_pool_view(h2o_pool* pool, int layer, void** K, void** V, float** k_scale, float** v_scale,
                  int32_t** pos, float** score, int32_t** table, int32_t** meta, int32_t** ref);

/*
 * h2o_pool_write - append tokens to sequences of one layer: a prompt, or the
 * next token(s) of a step. Entry i appends lens[i] tokens (T with lens NULL;
 * a length outside [0, T] is clamped and sets bit 4) from K, V, device bf16
 * [n][H][T][d], 16-byte aligned, with initial scores score, device fp32
 * [n][H][T] (a prompt's column sums from h2o_prefill_attention; NULL: zeros).
 * They take the sequence's next positions. With T = 0 K and V may be NULL: the
 * lists are checked alone. An entry that would grow beyond
 * max_pages is refused, unchanged, with bit 8.
 * Errors: H2O_EINVAL, H2O_ENOMEM, H2O_ECUDA.
 */
int h2o_pool_write(h2o_pool* pool, int layer, int n, const int32_t* seqs, const void* K,
                   const void* V, int T, const int32_t* lens, const float* score);

/*
 * h2o_pool_append - h2o_pool_write of a projection's output: keys are normed and
 * rotated at the positions that they take, on the way into the pages (rounded once,
 * to bf16 or to codes), and so are the queries (x->q, may be absent: q_heads is then
 * ignored) into q_out, bf16 [n][T][q_heads][d], 16-byte aligned, as h2o_pool_attend (T = 1)
 * and h2o_pool_attend_tree take them. x has n entries of T tokens; x->heads and
 * x->head_dim are the pool's. Scores begin at zero. lens, refusals and error bits as for
 * h2o_pool_write; rows of q_out that belong to no written token stay as they were.
 *
 * parent: the tokens are drafts, T <= H2O_POOL_MAX_NODES: device int32 [n][T], token t of
 * an entry hangs below parent[t] < t, or (-1) below the sequence's last token; one that is
 * no earlier token sets bit 16 and counts as -1. A draft's position is its depth further
 * than the next position, which stays until h2o_pool_accept. With parent NULL the tokens
 * follow each other and the next position moves on. Drafts are to be accepted or dropped
 * before the sequence is written, forked, copied, compacted or attended to otherwise.
 *
 * A round goes on without a look at the error word: while the last tokens that were to
 * be written to a sequence, by this call or by h2o_pool_write, were refused,
 * h2o_pool_attend_tree and h2o_pool_accept pass over its entries as over -1 (what it
 * holds is no drafts), and, where this call had queries, so does h2o_pool_attend (their
 * rows were not written). It ends, layer by layer, with a write or append that is
 * served, a fork or copy into the sequence, h2o_pool_free or h2o_pool_accept.
 * Errors: H2O_EINVAL, H2O_ENOMEM, H2O_ECUDA.
 */
int h2o_pool_append(h2o_pool* pool, int layer, int n, const int32_t* seqs, const h2o_qkv* x,
                    const h2o_rotary* rotary, int T, const int32_t* lens, const int32_t* parent,
                    void* q_out);

/*
 * h2o_pool_fork - make the empty sequence dst[i] a continuation of src[i]
 * (layer -1: in every layer): it shares the whole pages, gets a copy of the
 * partial last page (at most one fresh page), and its own copy of the scores.
 * h2o_pool_copy - the same with every page copied: nothing is shared.
 * A dst that is not empty sets bit 16 and is skipped. Sources are read as they
 * were before the call. Errors: H2O_EINVAL, H2O_ENOMEM, H2O_ECUDA.
 */
int h2o_pool_fork(h2o_pool* pool, int layer, int n, const int32_t* src, const int32_t* dst);
int h2o_pool_copy(h2o_pool* pool, int layer, int n, const int32_t* src, const int32_t* dst);

/*
 * h2o_pool_free - empty sequences (layer -1: in every layer): each of their
 * pages loses a holder, and is free when it had no other. Freeing an empty
 * sequence does nothing. Errors: H2O_EINVAL, H2O_ECUDA.
 */
int h2o_pool_free(h2o_pool* pool, int layer, int n, const int32_t* seqs);

/*
 * h2o_pool_compact - apply the policy to sequences (layer -1: in every layer):
 * each head of a sequence longer than h + r keeps the r last tokens and the h
 * others with the largest (score, position) keys, in ascending order, as
 * h2o_prefill selects from a prompt; shorter sequences are left as they are.
 * Scores order as fp32 values, NaN above all. The kept tokens move to
 * ceil((h + r) / page) fresh pages, so that other holders of the old pages keep
 * theirs; the old pages then lose a holder. The next position is unchanged.
 * h >= 0, r >= 0, 1 <= h + r <= H2O_MAX_K.
 * Errors: H2O_EINVAL, H2O_ENOMEM, H2O_ECUDA.
 */
int h2o_pool_compact(h2o_pool* pool, int layer, int n, const int32_t* seqs, int h, int r);

/*
 * h2o_pool_attend - attention of one query token per sequence of a batch over
 * the tokens of sequence `prefix` (-1: none), which all of them share and which
 * is read once for the batch, and over each sequence's own tokens. Write a
 * step's token first if it is to attend to itself.
 *
 * For row (i, query head hq), key head hq / (q_heads / H): p = softmax(q . k /
 * sqrt(d)) over both token lists, out = sum_j p_j v_j (bf16, rounded once from
 * an fp32 sum; p_j, in an H2O_KV_FP8 pool times v_j's scale, enters it with 16
 * significant bits, as two bf16 terms), lse = the natural log of the softmax's
 * normaliser (fp32; may be NULL). An H2O_KV_FP8 pool takes a query's values as two
 * E4M3 codes each: what is lost of a value is at most 2^-17 of the largest value of
 * its row, or 2^-136. Sums of p_j v_j are kept in units of the largest p_j so far,
 * up to 2^8: values beyond 2^120 divided by the number of tokens can leave fp32.
 * With accumulate, every probability is added to its slot's accumulated score:
 * to the sequence's for its own tokens (summed over the head's query group), to
 * the prefix's, summed over group and batch, for the prefix: the statistic by
 * which h2o_pool_compact can compact the prefix for all. Sums run in a fixed
 * order: equal calls give equal bits. Without any token out is 0 and lse is
 * -infinity. Rows of skipped entries keep what they held, as do those of entries whose
 * queries h2o_pool_append did not write.
 *
 * q: device bf16 [n][q_heads][d]; out: device bf16 [n][q_heads][d]; lse: device
 * fp32 [n][q_heads]; q and out 16-byte aligned; the three must not overlap.
 * q_heads is a multiple of H, at most H2O_POOL_MAX_GROUP times. `prefix` in `seqs`
 * is a bad entry. With accumulate the call's scratch holds 4 bytes per query row
 * and slot of a longest sequence, 4 n q_heads C (twice that for a prefix with at
 * most 32 rows a head). Where the allocator does not have that much the batch is
 * served in 2, 4, ... parts, each of which reads the prefix, and adds to its scores,
 * in its turn; H2O_ENOMEM when there is no memory for one entry.
 * Errors: H2O_EINVAL, H2O_ENOMEM, H2O_ECUDA.
 */
int h2o_pool_attend(h2o_pool* pool, int layer, int n, const int32_t* seqs, int prefix,
                    const void* q, int q_heads, void* out, float* lse, int accumulate);

/*
 * h2o_pool_attend_tree - attention of drafted tokens: the last lens[i] (device int32 [n];
 * NULL: T) tokens of sequence i are a tree's nodes, as h2o_pool_append (or a write) left
 * them. Row (i, t, query head) attends to the tokens of `prefix` (-1: none), to the
 * sequence's tokens before the nodes, to the nodes that node t hangs below and to itself;
 * else as h2o_pool_attend, without scores (h2o_pool_accept adds those of the rows that
 * were kept). Keys and values of other nodes, whatever they are, do not reach a row.
 * The prefix is read for every sequence: it costs as much as tokens of their own would.
 *
 * parent: device int32 [n][T] as for h2o_pool_append; NULL: each node hangs below the one
 * before it, the next tokens of a prompt for instance. q, out: device bf16
 * [n][T][q_heads][d], 16-byte aligned; lse: device fp32 [n][T][q_heads], may be NULL; the
 * three must not overlap. Rows t >= lens[i] and those of skipped entries keep what they
 * held; so do those of entries whose tokens were refused (h2o_pool_append). A length
 * outside [0, T] is clamped, and one beyond the sequence's skips the entry; both set bit 4.
 * 0 <= T <= H2O_POOL_MAX_NODES, n * T * q_heads < 2^31. Scratch: some 2^11 (d + 2) bytes an
 * SM (40 MB on 152 with d = 128), and 2 d + 4 more a row of q in an H2O_KV_FP8 pool.
 * Errors: H2O_EINVAL, H2O_ENOMEM, H2O_ECUDA.
 */
int h2o_pool_attend_tree(h2o_pool* pool, int layer, int n, const int32_t* seqs, int prefix,
                         const void* q, int q_heads, int T, const int32_t* lens,
                         const int32_t* parent, void* out, float* lse);

/*
 * h2o_pool_accept - keep some of the drafts, the last lens[i] (device int32 [n]; NULL: T)
 * tokens of each sequence, and drop the others (layer -1, without q: in every layer).
 * path: device int32 [n][P], the nodes that stay in ascending order, each below the one
 * before it, -1 behind the last (P = 0: none stays, path may be NULL). Kept tokens move
 * together behind the tokens before the drafts, with scores of zero; pages behind them
 * lose a holder. The next position becomes the first draft's plus the number of kept
 * ones. Pages that are written, or that become a partial last one, must be the
 * sequence's alone (they are, unless it was forked while it held drafts): else the entry
 * is refused, unchanged, with bit 2. A path that does not ascend or names no draft, and a
 * sequence that is `prefix`, set bit 16, and the entry is refused, unchanged; lengths as for
 * h2o_pool_attend_tree. An entry whose tokens were refused (h2o_pool_append) is passed over,
 * once.
 *
 * With q, device bf16 [n][T][q_heads][d], 16-byte aligned, and lse, device fp32
 * [n][T][q_heads], as h2o_pool_attend_tree took and gave them, the probabilities of the
 * kept rows are added to the accumulated scores: exp(q . k / sqrt(d) - lse) to every token
 * that the row attends to, the prefix's (-1: none) summed over the batch as h2o_pool_attend
 * with accumulate does for single tokens. Rows of no kept draft are not read. One with an
 * infinite lse adds nothing. Sums run in a fixed order: equal calls give equal bits. 0 <= T, P <=
 * H2O_POOL_MAX_NODES. Errors: H2O_EINVAL, H2O_ENOMEM, H2O_ECUDA.
 */
int h2o_pool_accept(h2o_pool* pool, int layer, int n, const int32_t* seqs, int T,
                    const int32_t* lens, const int32_t* path, int P, const void* q, int q_heads,
                    const float* lse, int prefix);

/* h2o_pool_sync_check - h2o_sync_check for a pool's error word. */
int h2o_pool_sync_check(h2o_pool* pool);

/* h2o_last_error - message of the calling thread's last failed call ("" if none). */
const char* h2o_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* H2O_H */
