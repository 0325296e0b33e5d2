/*
 * pa.h -- C ABI of the GB300 (sm_103a) paged-attention library.
 *
 * The library computes attention for decode and chunked-prefill queries over a KV cache stored
 * in fixed-size physical blocks reached through a per-sequence block table, with grouped-query
 * heads and prefix blocks that may be aliased across sequences:
 *   - "Local_LLM_03_vLLM_Architecture", paged-KV slide: fixed-size blocks (16 tokens by
 *     default), a per-sequence block table from logical positions to physical blocks, and an
 *     attention kernel that gathers K/V from the scattered blocks; block-size slide: the block
 *     size is a knob; KV-sizing slide: GQA-8; chunked-prefill slide: prefills cut into chunks
 *     and interleaved with decodes.
 *   - "vLLM: LLM Inference That Doesn't Waste Your GPU", sections "KV cache, in one picture"
 *     (every processed token's K/V is stored once and reused), "Continuous batching" (prefill and
 *     decode mixed in one step) and "PagedAttention: virtual memory for KV".
 *   - "Scaling inference with vLLM": requests with the same start share physical pages.
 *
 * Conventions (the pages fix none of them):
 *   - Every pointer in a pa_tensor is a DEVICE pointer of the current CUDA device.  The library
 *     owns no buffer and allocates no device memory; the caller owns everything, including
 *     the attention workspace.
 *   - Strides are in elements.  The innermost dimension must be contiguous (stride 1).
 *   - fp16 is IEEE binary16; bf16 is bfloat16 (the upper half of an IEEE binary32).  A call
 *     works in one 16-bit type: k, v, q, out and the pools all fp16 or all bf16 (FP8 pools take
 *     fp16 tokens, q and out).  Accumulation is fp32; outputs are rounded to nearest-even.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream), like a
 *     kernel launch.  Nothing synchronises except pa_get_device_error.
 *   - Host-checkable errors are returned synchronously and nothing is launched.  Device-data
 *     errors (a slot or block id outside the pool, query_len > seq_len, a sequence longer than
 *     the hint) make the affected work item skip its memory accesses, set a bit in a device
 *     error word (the device's, or the stream's own: pa_set_stream_error_word) and leave its
 *     output rows unwritten; pa_get_device_error reports them.
 *   - Every wait inside a kernel gives up after two seconds (pa_set_wait_limit) and reports
 *     PA_ERR_TIMEOUT.
 *   - Thread-safety: functions may be called from several host threads; pa_last_error is
 *     per thread.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PA_VERSION 3
#define PA_PARTITION_TOKENS 512 /* keys per split-context partition */
#define PA_MAX_DIMS 5

typedef enum pa_status {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1, /* bad pointer, dtype, rank, shape, stride or alignment */
  PA_ERR_UNSUPPORTED = 2, /* well-formed but not built: head_dim, block_size, group size */
  PA_ERR_CUDA = 3,        /* CUDA runtime error; pa_last_error() has the message */
  PA_ERR_TIMEOUT = 4,     /* device: a bounded wait gave up (reported by pa_get_device_error) */
  PA_ERR_OUT_OF_RANGE = 5,/* device: slot or block id outside the pool; access skipped */
  PA_ERR_WORKSPACE = 6,   /* workspace missing, misaligned or smaller than required */
  PA_ERR_DESCRIPTOR = 7,  /* device: query_len > seq_len, short block table, or hint exceeded */
  PA_ERR_NO_BLOCKS = 8    /* host block manager: too few free or evictable blocks */
} pa_status;

typedef enum pa_dtype {
  PA_F16 = 0,
  PA_I32 = 1,
  PA_I64 = 2,
  PA_F8E4M3 = 3, /* one byte: 1 sign, 4 exponent (bias 7), 3 mantissa bits; 0x7F/0xFF NaN, max 448 */
  PA_BF16 = 4,   /* bfloat16: 1 sign, 8 exponent (bias 127), 7 mantissa bits */
  PA_F32 = 5     /* IEEE binary32: weights of pa_diff_attention only */
} pa_dtype;

typedef struct pa_tensor {
  void* data;                 /* device pointer, 16-byte aligned for fp16 / bf16 tensors */
  int32_t dtype;              /* pa_dtype */
  int32_t ndim;
  int64_t shape[PA_MAX_DIMS];
  int64_t stride[PA_MAX_DIMS];/* in elements */
} pa_tensor;

/* Host-side facts about the batch the scheduler already knows.  Upper bounds are fine; a
 * sequence that exceeds them is skipped on the device and reported as PA_ERR_DESCRIPTOR. */
typedef struct pa_batch_hint {
  int32_t max_query_len;    /* max over sequences of query_start_loc[s+1] - query_start_loc[s] */
  int32_t max_seq_len;      /* max over sequences of seq_lens[s] */
  int32_t num_prefill_seqs; /* count of sequences with more than one query row; 0 = not known,
                               then the prefill launch covers every sequence.  A batch with more
                               such sequences than this skips the extra ones and reports
                               PA_ERR_DESCRIPTOR.  When it equals the number of sequences (and
                               max_query_len > 1) the decode launches are skipped; a one-row
                               sequence in such a batch is then reported the same way. */
  int32_t shared_prefix_tokens; /* 0, or a multiple of 512 (and of the block size) smaller than
                               every sequence's seq_len: the first shared_prefix_tokens keys of
                               every sequence are the same physical blocks (the block tables
                               agree there), so they are attended once for all query rows (p1:
                               requests that start alike share pages; p2 prefix-caching slide)
                               and merged with each sequence's own keys by the log-sum-exp rule.
                               Decode rows only (else PA_ERR_UNSUPPORTED); a
                               sequence whose table differs there, or with no key past the
                               prefix, is reported as PA_ERR_DESCRIPTOR. */
} pa_batch_hint;

/*
 * pa_reshape_and_cache -- write this step's new K/V tokens into their cache slots.
 * ("vLLM: LLM Inference That Doesn't Waste Your GPU", "KV cache, in one picture": the K/V of every
 * processed token is stored once; "Local_LLM_03_vLLM_Architecture", paged-KV slide: the store is a
 * set of fixed-size blocks.)
 *
 *   k, v          fp16 or bf16 [T_new, Hkv, d]; token stride free (multiple of 8), head stride d.
 *   k_cache,
 *   v_cache       [NB, Hkv, bs, d] of the same type as k and v, contiguous ("HND" per block: one (block, kv head) is a
 *                 contiguous bs x d tile).  Written in place.
 *   slot_mapping  int64 [T_new]; token t goes to block slot/bs, offset slot%bs.  slot < 0 means
 *                 "padding, skip".  A slot >= NB*bs is skipped and reported on the device.
 * For every t with slot >= 0 and every kv head h: k_cache[slot/bs][h][slot%bs][:] = k[t][h][:]
 * (bit-exact copy), same for v.  Two tokens with the same slot race (the last writer is
 * unspecified), as the pages give no order between them.
 * Supported: d in {64, 128}, bs in {16, 32}.
 */
int pa_reshape_and_cache(const pa_tensor* k, const pa_tensor* v, const pa_tensor* k_cache,
                         const pa_tensor* v_cache, const pa_tensor* slot_mapping, void* stream);

/*
 * pa_attention_workspace_size -- bytes of scratch pa_attention needs for a batch.
 * Split-context partials: for T query rows, Hq heads and P = ceil(max_seq_len / 512)
 * partitions, fp32 o[T][Hq][P][d] plus fp32 m[T][Hq][P] and l[T][Hq][P].  0 when P <= 1.
 */
size_t pa_attention_workspace_size(int64_t num_tokens, int64_t num_q_heads, int64_t head_dim,
                                   int32_t max_seq_len);

/*
 * pa_attention -- paged attention for one mixed continuous-batching step.
 * ("Local_LLM_03_vLLM_Architecture", paged-KV slide: the kernel gathers K/V from scattered
 * physical blocks through the block table; chunked-prefill slide; "vLLM: LLM Inference That
 * Doesn't Waste Your GPU", "Continuous batching": prefill and decode in the same step.)
 *
 *   q                fp16 or bf16 [T, Hq, d]; token stride free (multiple of 8), head stride d.
 *   k_cache, v_cache [NB, Hkv, bs, d] of q's type, contiguous, already holding this step's tokens
 *                    (call pa_reshape_and_cache first, on the same stream).
 *   block_tables     int32 [N, MB]; row stride free.  Entry j of row s = physical block of
 *                    logical positions j*bs .. j*bs+bs-1 of sequence s.  Entries past
 *                    ceil(seq_lens[s]/bs) are never read.  Aliasing (the same block id in
 *                    several rows) is allowed and is how shared prefixes are expressed.
 *   seq_lens         int32 [N]; keys of sequence s after this step's tokens were written.
 *   query_start_loc  int32 [N+1]; query_start_loc[0] = 0, non-decreasing, [N] = T.  Sequence s
 *                    owns rows query_start_loc[s] .. query_start_loc[s+1]-1.  One row is a
 *                    decode step, several a prefill chunk; any mix and order in one call.
 *   scale            multiplies q.k before the softmax (typically 1/sqrt(d)).
 *   out              [T, Hq, d] of q's type, contiguous.
 *   hint             required; see pa_batch_hint.
 *   workspace        device scratch of at least pa_attention_workspace_size(T, Hq, d,
 *                    hint->max_seq_len) bytes, 256-byte aligned (NULL allowed when that is 0).
 *                    Owned by the caller; must not be shared by calls in flight at once.
 * Row i of sequence s sits at absolute position seq_lens[s] - q_len + i and attends to keys
 * 0 .. seq_lens[s] - q_len + i (bottom-right causal; q_len = 1 attends to all keys).  Query
 * head h reads kv head h / (Hq / Hkv).  out = softmax(scale * q K^T) V per row and head.
 * Rows with q_len = 1 and more than 512 keys are computed in 512-key partitions merged with
 * the log-sum-exp rule; so are verify rows (every sequence with at most a few rows: q_len x G
 * <= 8, or <= 32 over an FP8 cache), each with its own causal limit.  Longer chunks run on the
 * tensor-core prefill kernels, beside the decode work when the call has both; the
 * shared-prefix pass (hint->shared_prefix_tokens) runs beside the decode kernel too.  Both use
 * a side stream of the library's (one per device and host thread, created by the first such
 * call), forked from and joined back into `stream` with events, so a capture of the call into a
 * CUDA graph records the fork and the join.
 * Supported: d in {64, 128}, bs in {16, 32}, Hq / Hkv in 1..16.
 */
int pa_attention(const pa_tensor* q, const pa_tensor* k_cache, const pa_tensor* v_cache,
                 const pa_tensor* block_tables, const pa_tensor* seq_lens,
                 const pa_tensor* query_start_loc, float scale, const pa_tensor* out,
                 const pa_batch_hint* hint, void* workspace, size_t workspace_bytes,
                 void* stream);

/*
 * FP8 KV cache ("Local_LLM_03_vLLM_Architecture", KV-sizing slide: the cache's bytes per token
 * decide how many sequences fit and how fast decode reads them; the pages quantise weights
 * only, so storing K/V in 8 bits is this library's extension).  The pools are PA_F8E4M3
 * [NB, Hkv, bs, d] with one scale per tensor: a stored code c of K stands for
 * k_scale * value(c), of V for v_scale * value(c).  Both scales must be finite and > 0.
 */
typedef struct pa_kv_scales {
  float k_scale;
  float v_scale;
} pa_kv_scales;

/*
 * pa_reshape_and_cache_fp8 -- pa_reshape_and_cache into an FP8 cache: each new value x (fp16)
 * is stored as the E4M3 code of x * (1 / scale), the reciprocal and the product in float32,
 * rounded to nearest even; magnitudes from 448 up (and infinities) saturate to +-448, NaN
 * stays NaN.  Arguments and errors as pa_reshape_and_cache, with k_cache / v_cache PA_F8E4M3.
 */
int pa_reshape_and_cache_fp8(const pa_tensor* k, const pa_tensor* v, const pa_tensor* k_cache,
                             const pa_tensor* v_cache, const pa_tensor* slot_mapping,
                             const pa_kv_scales* scales, void* stream);

/*
 * pa_attention_fp8 -- pa_attention over an FP8 cache (q and out stay fp16).  Every E4M3 value
 * is exact in fp16, so the kernels widen the codes to fp16 (decode: into MMA operands in
 * registers; prefill: tile by tile in shared memory) and run the fp16 arithmetic with the score
 * scale multiplied by k_scale and the output by v_scale.  Any mix of decode, verify and prefill
 * rows, and the shared-prefix pass, as for pa_attention.  Workspace as for pa_attention.
 */
int pa_attention_fp8(const pa_tensor* q, const pa_tensor* k_cache, const pa_tensor* v_cache,
                     const pa_tensor* block_tables, const pa_tensor* seq_lens,
                     const pa_tensor* query_start_loc, float scale, const pa_tensor* out,
                     const pa_batch_hint* hint, const pa_kv_scales* scales, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * pa_attention_static_scratch -- pa_attention without a caller-provided workspace, for callers
 * that cannot allocate device memory (no paper counterpart: the pages describe no such call).
 *
 * Some callers may not call cudaMalloc at all: plugins inside a host program whose own pool
 * owns all device memory, or code on a serving path where allocating is not allowed because
 * cudaMalloc may block or synchronise and cudaFree synchronises the device.  This call takes the
 * same arguments as pa_attention minus the workspace and uses a fixed 32 MiB array in the
 * library's device memory for the split-context partials instead.  It allocates nothing.
 *   - Every GPU that loads the library holds the 32 MiB until the process exits.
 *   - A batch needing more than 32 MiB of scratch (pa_attention_workspace_size(T, Hq, d,
 *     hint->max_seq_len) > 32 MiB) is rejected with PA_ERR_WORKSPACE and a message; nothing runs.
 *   - The first call on each device looks up the array's device address (cudaGetSymbolAddress,
 *     with that device current) and caches it; make that first call before any stream capture.
 *     The cached address belongs to the device's primary context as it was then: after
 *     cudaDeviceReset (or any teardown of that context) this entry point must not be called
 *     again in the same process.
 *   - All calls on a device share the array, which keeps the last call's contents; nothing in it
 *     needs to start at zero.  Calls that overlap on the GPU race on it: order them.
 * Results are those of pa_attention on the same inputs.
 */
int pa_attention_static_scratch(const pa_tensor* q, const pa_tensor* k_cache,
                                const pa_tensor* v_cache, const pa_tensor* block_tables,
                                const pa_tensor* seq_lens, const pa_tensor* query_start_loc,
                                float scale, const pa_tensor* out, const pa_batch_hint* hint,
                                void* stream);

/* Message for the last non-OK status returned on this host thread ("" if none). */
const char* pa_last_error(void);

/*
 * pa_get_device_error -- synchronise `stream`, then read and clear the error word that calls on
 * `stream` report into: the word registered for it with pa_set_stream_error_word, else the
 * current device's own word (shared by every unregistered stream of the device).  Returns PA_OK,
 * PA_ERR_TIMEOUT, PA_ERR_OUT_OF_RANGE or PA_ERR_DESCRIPTOR (most severe first); *bits (may be
 * NULL) receives the raw word: 1 timeout, 2 slot out of range, 4 block id out of range,
 * 8 descriptor, 16 hint exceeded.
 */
int pa_get_device_error(void* stream, uint32_t* bits);

/*
 * pa_set_stream_error_word -- let later calls on `stream` (a cudaStream_t; NULL is the legacy
 * default stream) report their device errors into `device_word` instead of the device's shared
 * word, so that a caller serving several streams reads each stream's errors apart.  The word is
 * a caller-owned, 4-byte aligned device uint32 that the caller zeroes first; the library only
 * ORs bits into it and pa_get_device_error(stream, ...) clears it.  NULL turns the stream back
 * to the device's word.  The word must stay allocated while calls registered to it can run.  At
 * most 64 streams hold a word of their own at a time (PA_ERR_INVALID_ARG beyond, and for a
 * misaligned word).  Any host thread may register; the registration is process-wide.
 */
int pa_set_stream_error_word(void* stream, uint32_t* device_word);

/*
 * pa_copy_blocks -- copy whole physical blocks of the pool: K and V of every kv head of block
 * pairs[i][0] are copied to block pairs[i][1] ("Local_LLM_03_vLLM_Architecture", prefix-caching
 * slide: shared blocks; a sequence that appends into a partial block it shares gets its own
 * copy first, the copy-on-write the host block manager asks for).
 *   k_cache, v_cache  [NB, Hkv, bs, d], contiguous, fp16, bf16 or PA_F8E4M3 (both the same).
 *   pairs             int32 [n, 2] contiguous device array (src, dst).  Destinations must be
 *                     distinct and never a source of the same call.
 * A pair with an id outside the pool is skipped and reported as PA_ERR_OUT_OF_RANGE by
 * pa_get_device_error.  n = 0 is a no-op.
 */
int pa_copy_blocks(const pa_tensor* k_cache, const pa_tensor* v_cache, const pa_tensor* pairs,
                   void* stream);

/*
 * pa_rope_and_cache -- rotary positions with one or several axes, and the step's K/V into their
 * slots: q is rotated into q_out, k rotated and v unchanged are written as pa_reshape_and_cache
 * writes them.  (No paper counterpart: the pages take rotated keys as given.)
 *
 * Of every q and k head, pair i < num_pairs turns by theta = positions[axis_of_pair[i]][t] *
 * inv_freq[i]: (a, b) -> factor * (a cos theta - b sin theta, b cos theta + a sin theta), where
 * (a, b) are dims (i, i + num_pairs), or (2i, 2i + 1) when `adjacent`.  Dims from 2 * num_pairs
 * on are copied.  Several axes are the time, height and width of an image or video token; text
 * gives every axis the same position.
 *   q               fp16 or bf16 [T, Hq, d]; token stride free (multiple of 8), head stride d.
 *   k, v            same type [T, Hkv, d], strides as q's.
 *   positions       int64 [A, T], A in 1..255; axis stride free.  Any value, also negative;
 *                   angles are exact to float32 for |position| < 2^31.
 *   rope            HOST struct and HOST arrays, read before the call returns.
 *   k_cache,v_cache [NB, Hkv, bs, d] of q's type, or PA_F8E4M3 (fp16 q, k, v) with scales: a
 *                   value's code is E4M3(x * (1 / scale)) of the unrounded rotated x.
 *   slot_mapping    int64 [T] as in pa_reshape_and_cache: negative slots write no K/V (q is
 *                   rotated all the same), slots past the pool are reported.
 *   q_out           [T, Hq, d] of q's type, strides as q's; q itself (in place) or memory that
 *                   overlaps neither q, k nor v.
 *   scales          required for PA_F8E4M3 pools, else ignored (may be NULL).
 * Arithmetic is float32 with one rounding per output.  Supported: d in {64, 128}, bs in
 * {16, 32}, num_pairs a multiple of 8 up to d / 2.
 */
typedef struct pa_rope {
  int32_t num_pairs;           /* R / 2 rotated pairs per head */
  int32_t adjacent;            /* 0: pair (i, i + num_pairs); 1: pair (2i, 2i + 1) */
  float factor;                /* multiplies cos and sin (1 normally) */
  const double* inv_freq;      /* [num_pairs] radians per position */
  const int32_t* axis_of_pair; /* [num_pairs] axis of each pair; NULL: axis 0 for all */
} pa_rope;

int pa_rope_and_cache(const pa_tensor* q, const pa_tensor* k, const pa_tensor* v,
                      const pa_tensor* positions, const pa_rope* rope, const pa_tensor* k_cache,
                      const pa_tensor* v_cache, const pa_tensor* slot_mapping,
                      const pa_tensor* q_out, const pa_kv_scales* scales, void* stream);

/*
 * pa_diff_attention -- differential attention for one mixed continuous-batching step: the
 * difference of two softmax maps with learned weights, over the same pools, tables and batch
 * description as pa_attention.  (No paper counterpart.)
 *
 * Heads come in pairs: q heads 2p and 2p + 1 are the queries of the two maps of differential head
 * p; K heads 2j and 2j + 1 hold the two maps' keys and V heads 2j, 2j + 1 the halves of one
 * 2d-wide value, j = p / (Hq / Hkv).  For each row, over the keys it sees in pa_attention:
 *   y = softmax(scale q_2p K_2j^T) [V_2j | V_2j+1] - lambda_p softmax(scale q_2p+1 K_2j+1^T) [...]
 *   out = out_scale * y * rsqrt(mean(y^2) + eps) * norm_weight     (without norm_weight:
 *   out = out_scale * y)
 *   q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, hint, workspace
 *                    as in pa_attention, with Hkv (and so Hq) even, fp16 or bf16;
 *                    hint->shared_prefix_tokens must be 0.
 *   diff->lambda     float32 [Hq / 2], or [T, Hq / 2] (token stride free): one per token and head.
 *   diff->norm_weight float32 [2d] or NULL.
 *   out              [T, Hq / 2, 2d] of q's type, contiguous.
 *   workspace        device scratch of pa_diff_attention_workspace_size(...) bytes for the same
 *                    tokens (T), sequences (N), heads and hint; 256-byte aligned.
 * Rows of sequences that the device finds invalid are left unwritten and reported, as in
 * pa_attention.  Accumulation is float32; a row's result depends on the batch's sizes (how its keys
 * are split) to rounding, not on other rows or on page order.  The weights of a row's hidden keys are 0, but a V value of NaN or infinity at a
 * key that some row of the same chunk sees may reach the chunk's other rows (0 * infinity).
 * Supported: d in {64, 128}, bs in {16, 32}, Hq / Hkv in 1..16; not over FP8 pools.
 */
typedef struct pa_diff {
  const pa_tensor* lambda;
  const pa_tensor* norm_weight; /* NULL: no norm */
  float eps;                    /* >= 0 */
  float out_scale;
} pa_diff;

/* 0 also for heads that the call refuses. */
size_t pa_diff_attention_workspace_size(int64_t num_tokens, int64_t num_seqs, int64_t num_q_heads,
                                        int64_t num_kv_heads, int64_t head_dim,
                                        const pa_batch_hint* hint);

int pa_diff_attention(const pa_tensor* q, const pa_tensor* k_cache, const pa_tensor* v_cache,
                      const pa_tensor* block_tables, const pa_tensor* seq_lens,
                      const pa_tensor* query_start_loc, float scale, const pa_diff* diff,
                      const pa_tensor* out, const pa_batch_hint* hint, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * pa_move_blocks -- move whole physical blocks inside the pool, in place, and give block tables
 * their new ids: the device side of a compaction (pa_bm_compact), in which a block may move into
 * one that moves on itself (chains and cycles, which pa_copy_blocks does not take).
 *
 * pa_move_plan_create takes n HOST pairs (src, dst): no two moves out of one block, no two into
 * one block, ids inside the pool; src = dst is no move.  NULL on error (pa_last_error).  The plan
 * holds no device memory and serves any number of pools of num_blocks blocks.
 *   k_cache, v_cache  [NB, Hkv, bs, d], or all layers at once: [L, NB, Hkv, bs, d] (each layer
 *                     contiguous, layer stride free), fp16, bf16 or PA_F8E4M3.
 *   block_tables      int32 [N, MB] (row stride free) or NULL: every entry that is a moved
 *                     block's old id becomes its new id; other entries, ids outside the pool
 *                     among them, stay.  Pass it with one call where pools are moved by several.
 *   workspace         pa_move_blocks_workspace_size(plan, k_cache, 1, block_tables != NULL) bytes
 *                     at least, 256-byte aligned (NULL allowed when that is 0); with room for
 *                     more layers, more are moved per launch.
 * After the call, block dst holds what block src held before it, for every pair; a block that
 * only moved out keeps its old content.  pa_move_plan_staged: blocks that pass through the
 * workspace (0 unless long chains or cycles meet).
 */
typedef struct pa_move_plan pa_move_plan;
pa_move_plan* pa_move_plan_create(const int32_t* pairs, int64_t n, int64_t num_blocks);
void pa_move_plan_destroy(pa_move_plan* plan);
int64_t pa_move_plan_staged(const pa_move_plan* plan);
size_t pa_move_blocks_workspace_size(const pa_move_plan* plan, const pa_tensor* k_cache,
                                     int32_t layers, int32_t with_tables);
int pa_move_blocks(const pa_move_plan* plan, const pa_tensor* k_cache, const pa_tensor* v_cache,
                   const pa_tensor* block_tables, void* workspace, size_t workspace_bytes,
                   void* stream);

/*
 * pa_set_timing_events -- measurement hook.  When both are non-NULL (cudaEvent_t handles),
 * every later pa_attention call on this host thread records `start` on its stream just before
 * launching the selected kernel and `stop` just after it, so a caller can time that kernel with
 * CUDA events inside a longer step: `kernel` is PA_TIMED_DECODE (the decode-partition kernel,
 * launched by every call with rows), PA_TIMED_PREFILL (the chunked-prefill kernel, launched
 * when hint->max_query_len > 1) or PA_TIMED_SHARED_PREFIX (the shared-prefix pass, launched
 * when hint->shared_prefix_tokens > 0).  No work is skipped or reordered.  Pass NULL, NULL to turn
 * the selected hook off.  Returns PA_OK, or PA_ERR_INVALID_ARG for an unknown `kernel`.
 */
#define PA_TIMED_DECODE 0
#define PA_TIMED_PREFILL 1
#define PA_TIMED_SHARED_PREFIX 2
int pa_set_timing_events(int kernel, void* start, void* stop);

/*
 * pa_set_wait_limit -- how long every bounded wait inside the kernels of later pa_attention and
 * pa_attention_fp8 calls on this host thread may last before it gives up: the waiting work item
 * then lets its own copies in flight land, leaves its output rows unwritten and sets the
 * timeout bit that pa_get_device_error reports as PA_ERR_TIMEOUT (the CUDA context stays
 * usable).  A legitimate wait lasts microseconds; the default is 2 s.  Returns PA_OK, or
 * PA_ERR_INVALID_ARG (limit unchanged) outside [PA_WAIT_LIMIT_MIN_NS, PA_WAIT_LIMIT_MAX_NS].
 */
#define PA_WAIT_LIMIT_DEFAULT_NS 2000000000ull
#define PA_WAIT_LIMIT_MIN_NS 1000ull
#define PA_WAIT_LIMIT_MAX_NS 10000000000ull
int pa_set_wait_limit(uint64_t limit_ns);

/* PA_VERSION of the built library. */
int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
