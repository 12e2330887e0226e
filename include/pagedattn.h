/*
 * pagedattn.h -- C ABI of libpagedattn.so, attention over a paged KV cache on
 * one NVIDIA GB300 (sm_103a).
 *
 * The four operations are the per-layer GPU hot path of a Nano-vLLM-style
 * serving engine, as described on these pages:
 *   [LIFE] "一个 prompt 的一生：nano-vllm 从起服务到吐出 token" (violet-quartz.github.io)
 *   [UML]  the Nano-vLLM walk-through at uml.org.cn
 *   [SRC2] "《Nano-vLLM源码逐行解析》第2篇 sequence.py、scheduler.py" (yeyulingfeng.com)
 *
 * Data layout (all row-major, contiguous):
 *   k_cache, v_cache  [num_blocks, block_size, num_kv_heads, head_dim] bf16: one
 *                     layer's view of the KV pool ([LIFE] §2.2.3; [UML] §3.2).
 *                     A slot s is row s of the pool viewed as
 *                     [num_blocks*block_size, num_kv_heads, head_dim].
 *   block_tables      [batch, max_blocks_per_seq] int32: logical block i of a
 *                     sequence -> physical block id ([UML] §1 Step2, §3.2).
 *                     Entries past a sequence's last block are never read.
 *   q                 [tokens, num_q_heads, head_dim] bf16; k, v [tokens,
 *                     num_kv_heads, head_dim] bf16 ([UML] §3.2 formats).
 *   Grouped-query attention: q head h reads kv head h / (num_q_heads/num_kv_heads).
 *
 * Ownership: every pointer argument is caller-owned memory; the library keeps
 * no pointer past the call, allocates nothing and never synchronises.  Device
 * pointers must be device memory of the current CUDA device.  All work is
 * enqueued on `stream` (a cudaStream_t passed as void*; NULL = legacy default
 * stream) and runs asynchronously.
 *
 * Errors, two kinds:
 *   - the return value: PKV_OK (0) or a negative PKV_ERR_* code for a problem
 *     the host can see (null pointer, bad size, unsupported head_dim,
 *     misaligned pointer, workspace too small, launch failure).  Nothing is
 *     enqueued when a call returns an error.
 *   - `status`: an optional device uint32 into which kernels OR the
 *     PKV_STATUS_* bits of data-dependent problems (a slot or block id outside
 *     the pool, a bad context length, ...).  The offending item is skipped
 *     (its outputs are zeros where the entry point says so); nothing traps.
 *     The caller clears the word; NULL disables reporting.
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PKV_API __attribute__((visibility("default")))
#else
#define PKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* ---- return codes ------------------------------------------------------ */
#define PKV_OK                        0
#define PKV_ERR_NULL_POINTER         -1
#define PKV_ERR_BAD_DIMENSION        -2
#define PKV_ERR_UNSUPPORTED_HEAD_DIM -3
#define PKV_ERR_MISALIGNED           -4
#define PKV_ERR_WORKSPACE_TOO_SMALL  -5
#define PKV_ERR_CUDA                 -6
#define PKV_ERR_UNSUPPORTED          -7

/* ---- device status bits ------------------------------------------------ */
#define PKV_STATUS_SLOT_OUT_OF_RANGE  (1u << 0) /* kv_store: slot >= num_blocks*block_size   */
#define PKV_STATUS_BAD_BLOCK_ID       (1u << 1) /* a block table entry outside [0,num_blocks) */
#define PKV_STATUS_BAD_CONTEXT_LEN    (1u << 2) /* context len < 0, > table capacity or > max */
#define PKV_STATUS_BAD_SEQLENS        (1u << 3) /* cu_seqlens not monotone, Lk < Lq, ...       */
#define PKV_STATUS_BAD_TEMPERATURE    (1u << 4) /* sample: temperature not positive & finite  */
#define PKV_STATUS_NO_FINITE_KEY      (1u << 5) /* sample: every key of a row is NaN           */
#define PKV_STATUS_WORKSPACE_OVERFLOW (1u << 6) /* more work items than the workspace holds   */
#define PKV_STATUS_WAIT_TIMEOUT       (1u << 7) /* a bounded in-kernel wait gave up           */
#define PKV_STATUS_BAD_SCALE          (1u << 8) /* an e4m3 cache's scale cannot be used        */
#define PKV_STATUS_BAD_TOKEN_ID       (1u << 9) /* logit rules: a token id >= vocab            */
#define PKV_STATUS_BAD_PENALTY        (1u << 10) /* logit rules: a penalty is not usable       */
#define PKV_STATUS_NO_ALLOWED_TOKEN   (1u << 11) /* logit rules: a row's mask leaves nothing   */

/* One layer's KV cache geometry: k_cache/v_cache are [num_blocks, block_size,
 * num_kv_heads, head_dim] bf16. */
typedef struct pkv_cache_desc {
    int32_t num_blocks;
    int32_t block_size;
    int32_t num_kv_heads;
    int32_t head_dim;
} pkv_cache_desc;

/* Library version, major*10000 + minor*100 + patch. */
PKV_API int pkv_version(void);

/* Text for a PKV_ERR_* return code (static storage). */
PKV_API const char* pkv_error_string(int code);

/* Text naming the lowest PKV_STATUS_* bit set in `bits` ("ok" for 0). */
PKV_API const char* pkv_status_string(uint32_t bits);

/*
 * Diagnostics (no counterpart on the pages).  Every in-kernel wait on a
 * shared-memory barrier polls at most `polls` times, then gives up: the kernel
 * sets PKV_STATUS_WAIT_TIMEOUT, lets the copies and tensor-core operations it
 * already issued finish, frees what it holds and returns (its outputs are then
 * unspecified).  The setting is process-wide and applies to calls enqueued
 * after it.  The default, PKV_DEFAULT_WAIT_POLLS, is far beyond any wait of a
 * healthy kernel; 0 makes every such wait give up at once, which is how the
 * tests exercise the unwinding path.  Returns PKV_OK.
 */
#define PKV_DEFAULT_WAIT_POLLS (1u << 20)
PKV_API int pkv_set_wait_poll_limit(uint32_t polls);

/*
 * kv_store -- the per-layer KV cache write ("store_kvcache").
 * [UML] §2.4 (KV written into the cache before attention), §1 Step2 (slot =
 * blockID*blockSize + loc); [LIFE] §3.3.2 / §4 (slot_mapping holds one
 * physical slot per flattened token, so the writer needs no paging logic).
 *
 *   k, v           device, [num_tokens, num_kv_heads, head_dim] bf16, 16-byte aligned
 *   k_cache/v_cache device, the pool, written in place, 16-byte aligned
 *   slot_mapping   device, [num_tokens] int32; slot < 0 skips the token (padding
 *                  rows of a fixed-shape batch); slot >= num_blocks*block_size
 *                  sets PKV_STATUS_SLOT_OUT_OF_RANGE and skips it
 * Row i of k and of v is copied bit for bit into slot slot_mapping[i].  The
 * slots of a call are to be different: rows are stored in 16-byte pieces in no
 * order, so that a slot of two tokens ends with pieces of both
 * (pkv_qk_norm_rope_kv_store and pkv_kv_store_fp8 store the last token's row).
 * Needs num_kv_heads*head_dim*2 to be a multiple of 16.  num_tokens == 0 is a
 * no-op.
 */
PKV_API int pkv_kv_store(const void* k, const void* v, void* k_cache, void* v_cache,
                 const int32_t* slot_mapping, int32_t num_tokens,
                 pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * Bytes of device workspace pkv_paged_decode needs for these sizes (a pure
 * host function; the same arguments give the same answer).  The split into
 * key chunks depends on the batch, so the size is not monotone in it: a
 * workspace shared by several batch sizes (e.g. one CUDA graph per size)
 * must be as large as the largest of their answers.
 */
PKV_API size_t pkv_paged_decode_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                        int32_t max_context_len, pkv_cache_desc cache);

/*
 * paged_decode -- decode attention, one query token per sequence, K/V read
 * through the block table ([UML] §2.4: the decode attention op; §3.2: Q as
 * (batch, 1, heads, head_dim), cache_seqlens, block_tables).
 *
 *   q             device, [batch, num_q_heads, head_dim] bf16
 *   k_cache/v_cache device, the pool (read only)
 *   block_tables  device, [batch, max_blocks_per_seq] int32
 *   context_lens  device, [batch] int32: keys of sequence b are its logical
 *                 positions 0..context_lens[b]-1 (the new token's K/V must
 *                 already be stored).  0 gives a zero output row.  A value < 0,
 *                 > max_blocks_per_seq*block_size or > max_context_len sets
 *                 PKV_STATUS_BAD_CONTEXT_LEN and gives zeros.
 *   max_context_len host upper bound of context_lens, sizes the split-KV grid
 *   scale         softmax scale (e.g. 1/sqrt(head_dim))
 *   out           device, [batch, num_q_heads, head_dim] bf16
 *   workspace     device, >= pkv_paged_decode_workspace_bytes(...) bytes,
 *                 16-byte aligned; holds the split-KV partial results
 * out[b,h] = sum_j softmax_j(scale * q[b,h].K_j) V_j, fp32 accumulation.
 * head_dim 64 or 128; num_q_heads a multiple of num_kv_heads.
 */
PKV_API int pkv_paged_decode(const void* q, const void* k_cache, const void* v_cache,
                     const int32_t* block_tables, int32_t max_blocks_per_seq,
                     const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
                     int32_t max_context_len, float scale, void* out,
                     void* workspace, size_t workspace_bytes,
                     pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * paged_decode split into a plan and a run, for a caller that attends many
 * layers over the same sequences: in a model's decode step every layer has the
 * same context_lens and block_tables, so the chunk schedule is the same for
 * all of them.  (No counterpart on the pages: it divides pkv_paged_decode's
 * work; the result is the same.)
 *
 * pkv_paged_decode_plan checks context_lens (a length outside
 * [0, min(max_context_len, max_blocks_per_seq * block_size)] sets
 * PKV_STATUS_BAD_CONTEXT_LEN and that sequence attends to nothing) and writes
 * the chunk schedule into the workspace.  pkv_paged_decode_run then attends with
 * it: the split-KV and combine kernels only.  A run must get the same
 * context_lens contents, batch, num_q_heads, max_context_len,
 * max_blocks_per_seq, cache geometry and workspace as the plan it follows, and
 * the plan must be enqueued earlier on the same stream (or have completed).  Any
 * number of runs may follow one plan; a run overwrites the workspace's partial
 * results, so runs sharing a workspace must not overlap.  Arguments have the
 * meaning they have in pkv_paged_decode.
 */
PKV_API int pkv_paged_decode_plan(const int32_t* context_lens, int32_t batch,
                                  int32_t num_q_heads, int32_t max_context_len,
                                  int32_t max_blocks_per_seq, void* workspace,
                                  size_t workspace_bytes, pkv_cache_desc cache,
                                  uint32_t* status, void* stream);
PKV_API int pkv_paged_decode_run(const void* q, const void* k_cache, const void* v_cache,
                                 const int32_t* block_tables, int32_t max_blocks_per_seq,
                                 const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
                                 int32_t max_context_len, float scale, void* out, void* workspace,
                                 size_t workspace_bytes, pkv_cache_desc cache, uint32_t* status,
                                 void* stream);

/*
 * paged_decode without a caller-provided workspace.  (Not an operation of the
 * pages: it exists for callers that cannot allocate device memory where they
 * call -- e.g. a plugin inside a host engine that owns and budgets all device
 * memory up front, or a latency-critical loop that must not pay for
 * cudaMalloc's implicit device-wide synchronisation.)
 *
 * Same arguments and results as pkv_paged_decode, minus workspace and
 * workspace_bytes.  The split-KV scratch is a fixed array of
 * PKV_STATIC_DECODE_WORKSPACE_BYTES compiled into the library; every GPU that
 * loads the library holds it until the process exits.  The call allocates
 * nothing (no cudaMalloc, no allocating library routine).
 *   - When pkv_paged_decode_workspace_bytes(batch, num_q_heads,
 *     max_context_len, cache) exceeds PKV_STATIC_DECODE_WORKSPACE_BYTES the
 *     call returns PKV_ERR_WORKSPACE_TOO_SMALL and enqueues nothing.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - All calls share the one array, which keeps the last call's contents
 *     (the kernels write every scratch entry they read, so no state carries
 *     over).  Calls that may overlap on the GPU -- on different streams, or
 *     from different host threads -- race on it: serialise them.
 */
#define PKV_STATIC_DECODE_WORKSPACE_BYTES (16u * 1024u * 1024u)
PKV_API int pkv_paged_decode_static_workspace(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t batch,
    int32_t num_q_heads, int32_t max_context_len, float scale, void* out,
    pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * kv_store then paged_decode, enqueued as one call: the per-layer pair the
 * engine runs every decode step ([LIFE] §2.2.4: store_kvcache, then the
 * attention op; [UML] §2.4).  Arguments are those of pkv_kv_store (k, v,
 * slot_mapping, num_tokens) followed by those of pkv_paged_decode; k_cache
 * and v_cache are written by the store and read by the decode.  The store and
 * the decode's set-up (its chunk schedule) run as one grid, so the pair costs
 * one launch and the longer of the two; the attention kernels wait for that
 * whole grid, so they read the stored rows whatever slots slot_mapping names.
 * Arguments are all checked before anything is enqueued.
 */
PKV_API int pkv_kv_store_paged_decode(
    const void* k, const void* v, const int32_t* slot_mapping, int32_t num_tokens,
    const void* q, void* k_cache, void* v_cache, const int32_t* block_tables,
    int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t batch,
    int32_t num_q_heads, int32_t max_context_len, float scale, void* out, void* workspace,
    size_t workspace_bytes, pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * One layer's k_cache / v_cache inside the whole KV pool the engine allocates
 * once, [2, num_layers, num_blocks, block_size, num_kv_heads, head_dim] bf16
 * ([LIFE] §2.2.3: kv_cache[0, l] and kv_cache[1, l] are views, not copies).
 * Pure host pointer arithmetic; nothing is read or enqueued.
 */
PKV_API int pkv_layer_cache(const void* kv_pool, int32_t num_layers, int32_t layer,
                            pkv_cache_desc cache, const void** k_cache, const void** v_cache);

/*
 * Bytes of device workspace pkv_paged_prefill_varlen needs (pure host function).
 */
PKV_API size_t pkv_paged_prefill_workspace_bytes(int32_t batch, int32_t total_q,
                                         int32_t num_q_heads, pkv_cache_desc cache);

/*
 * paged_prefill_varlen -- causal prefill over a flattened batch of
 * variable-length sequences whose first tokens may already be in the cache
 * (prefix caching, chunked prefill).  [UML] §2.4 and §3.2 (the varlen prefill
 * attention op: cu_seqlens_q/k, max_seqlen_q/k, block_tables when a prefix is
 * cached); [LIFE] §3.1 / [SRC2] Sequence walkthrough (a round computes
 * num_scheduled_tokens tokens starting at num_cached_tokens).
 *
 *   q             device, [total_q, num_q_heads, head_dim] bf16
 *   k, v          device, [total_q, num_kv_heads, head_dim] bf16: this call's
 *                 own keys/values, one row per query token
 *   k_cache/v_cache device, the pool (read only)
 *   cu_seqlens_q/k device, [batch+1] int32 prefix sums.  Sequence b has
 *                 Lq = cu_q[b+1]-cu_q[b] queries and Lk = cu_k[b+1]-cu_k[b] keys.
 *                 Keys j < Lk-Lq (the cached prefix) are read from the cache
 *                 through block_tables[b]; keys j >= Lk-Lq are rows
 *                 cu_q[b]+j-(Lk-Lq) of k/v.  Query i sits at position Lk-Lq+i
 *                 and attends keys j <= Lk-Lq+i (bottom-right causal).
 *   max_seqlen_q/k host upper bounds of Lq/Lk
 *   block_tables  device [batch, max_blocks_per_seq] int32, or NULL when no
 *                 sequence has a cached prefix (then Lk must equal Lq)
 *   scale         softmax scale, positive and finite (e.g. 1/sqrt(head_dim))
 *   out           device, [total_q, num_q_heads, head_dim] bf16
 *   workspace     device, >= pkv_paged_prefill_workspace_bytes(...) bytes,
 *                 16-byte aligned; holds the tile schedule
 * A sequence with inconsistent lengths sets PKV_STATUS_BAD_SEQLENS and is
 * skipped (its output rows are not written).  head_dim 64 or 128, any
 * block_size.  Entries of V are to stay below 2^96 in size: the sums before the
 * softmax's division may stand 2^32 above them.  PKV_ERR_UNSUPPORTED:
 * num_blocks*block_size >= 2^31 (no such pool fits in device memory) or a
 * driver without cuTensorMapEncodeTiled.
 */
PKV_API int pkv_paged_prefill_varlen(const void* q, const void* k, const void* v,
                             const void* k_cache, const void* v_cache,
                             const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                             int32_t batch, int32_t total_q, int32_t max_seqlen_q,
                             int32_t max_seqlen_k, int32_t num_q_heads,
                             const int32_t* block_tables, int32_t max_blocks_per_seq,
                             float scale, void* out, void* workspace, size_t workspace_bytes,
                             pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * kv_store followed by paged_prefill_varlen on the same stream: the per-layer
 * pair of a prefill round, cache write then attention ([LIFE] §2.2.4 and §4
 * store_kvcache before the attention op; [UML] §2.4).  The store writes this
 * call's k/v rows (total_q of them) to slot_mapping's slots (negative =
 * padding, skipped); the other arguments are those of
 * pkv_paged_prefill_varlen, with k_cache/v_cache written by the store and
 * required even when block_tables is NULL.  The prefill's tile plan is launched
 * as a programmatic dependent of the store, and the attention reads nothing
 * until both are done.  Every argument is checked before anything is
 * enqueued.
 */
PKV_API int pkv_kv_store_paged_prefill_varlen(
    const void* q, const void* k, const void* v, void* k_cache, void* v_cache,
    const int32_t* slot_mapping, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
    int32_t batch, int32_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k,
    int32_t num_q_heads, const int32_t* block_tables, int32_t max_blocks_per_seq, float scale,
    void* out, void* workspace, size_t workspace_bytes, pkv_cache_desc cache, uint32_t* status,
    void* stream);

/*
 * Bytes of device workspace pkv_kv_store_paged_attention_varlen needs (pure
 * host function): the prefill's tile schedule followed by the decode's chunk
 * plan and partial results, the latter sized for max_seqlen_k keys.
 */
PKV_API size_t pkv_paged_attention_varlen_workspace_bytes(int32_t batch, int32_t total_q,
                                                  int32_t num_q_heads, int32_t max_seqlen_k,
                                                  pkv_cache_desc cache);

/*
 * kv_store then attention over a mixed batch: prefill chunks and decode
 * tokens in one step.  The pages' scheduler never mixes the two ([LIFE] §3.2),
 * but a step's sequences each compute num_scheduled_tokens tokens from
 * num_cached_tokens on ([LIFE] §3.1), so a decode row is a chunk of one token
 * and continuous batching ([UML] §2.1) can take both in one call.  The
 * arguments and the result are those of pkv_kv_store_paged_prefill_varlen
 * (bottom-right causal attention of every query row), computed in two passes:
 * sequences with Lq != 1 by the varlen prefill kernels, sequences with Lq == 1
 * by the split-KV decode kernels.  The second pass reads all Lk keys of a
 * one-query sequence from the cache through block_tables[b], its own key
 * included, so slot_mapping must store that row at position Lk-1 of
 * block_tables[b] (as an engine's slot mapping does); block_tables and the
 * cache are required.
 *   workspace     device, >= pkv_paged_attention_varlen_workspace_bytes(...)
 *                 bytes, 16-byte aligned
 * A one-query sequence whose lengths are inconsistent (Lk < 1, its row outside
 * q, more keys than max_seqlen_k or than its table holds) sets
 * PKV_STATUS_BAD_SEQLENS and its output row is not written.  Every argument
 * is checked before anything is enqueued.
 */
PKV_API int pkv_kv_store_paged_attention_varlen(
    const void* q, const void* k, const void* v, void* k_cache, void* v_cache,
    const int32_t* slot_mapping, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
    int32_t batch, int32_t total_q, int32_t max_seqlen_q, int32_t max_seqlen_k,
    int32_t num_q_heads, const int32_t* block_tables, int32_t max_blocks_per_seq, float scale,
    void* out, void* workspace, size_t workspace_bytes, pkv_cache_desc cache, uint32_t* status,
    void* stream);

/*
 * sample -- temperature, softmax and Gumbel-max sampling of one token per row
 * ([UML] §2.4: "温度、softmax和gumbel max"; [LIFE] §4: the sampler runs on each
 * sequence's last-position logits).  With supplied Exp(1) noise E the draw is
 * argmax_i softmax(logits/T)_i / E_i, computed as the equal
 * argmax_i (logits_i/T - ln max(E_i, 1e-10)); ties go to the lowest index.
 *
 *   logits        device, [batch, vocab] fp32
 *   temperatures  device, [batch] fp32; a value that is not positive and finite
 *                 sets PKV_STATUS_BAD_TEMPERATURE and the row returns 0
 *   exp_noise     device, [batch, vocab] fp32 Exp(1) draws
 *   out_token_ids device, [batch] int32
 * NaN keys never win; a row of NaN keys returns 0 and sets
 * PKV_STATUS_NO_FINITE_KEY.
 */
PKV_API int pkv_sample(const float* logits, const float* temperatures, const float* exp_noise,
               int32_t batch, int32_t vocab, int32_t* out_token_ids,
               uint32_t* status, void* stream);

/*
 * sample with the Exp(1) noise drawn inside the kernel instead of read from
 * memory (halves the sampler's HBM bytes).  The noise of entry n = row*vocab+i
 * comes from Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
 * numbers: as easy as 1, 2, 3", SC 2011) with key = seed (low word first) and
 * counter = (n/4 low, n/4 high, offset low, offset high), output word n%4:
 * U = ((w >> 8) + 1) * 2^-24 in (0, 1], E = -ln U.  Everything else is as in
 * pkv_sample (temperature, lowest-index ties, status bits).  The same (seed,
 * offset) gives the same draw; advance `offset` per step for fresh noise.
 */
PKV_API int pkv_sample_philox(const float* logits, const float* temperatures, uint64_t seed,
                              uint64_t offset, int32_t batch, int32_t vocab,
                              int32_t* out_token_ids, uint32_t* status, void* stream);

/*
 * ---- an 8-bit KV cache ---------------------------------------------------
 * (No counterpart on the pages, whose cache is bf16: half the cache bytes of
 * a decode step and twice the tokens in the same memory.)
 *
 *   k_cache, v_cache  [num_blocks, block_size, num_kv_heads, head_dim] e4m3
 *                     codes (1 sign, 4 exponent, 3 fraction bits, largest 448)
 *   k_scale, v_scale  [num_blocks, num_kv_heads] fp32: an entry's value is its
 *                     code times the scale of its block and kv head
 * block_size is at most PKV_FP8_MAX_BLOCK_SIZE, head_dim 64 or 128.  Attention
 * takes any scale in [2^-96, FLT_MAX].  A scale outside it (0 marks a block
 * without rows) sets PKV_STATUS_BAD_SCALE where a key needs it.
 */
#define PKV_FP8_MAX_BLOCK_SIZE 1024

/*
 * Bytes of device workspace pkv_kv_store_fp8 needs (a pure host function; 0
 * for small calls, which may pass a NULL workspace).
 */
PKV_API size_t pkv_kv_store_fp8_workspace_bytes(int32_t num_tokens, pkv_cache_desc cache);

/*
 * kv_store into an e4m3 cache.  Arguments as in pkv_kv_store (k, v bf16), with
 * the cache's scales read and written.  For each (block, kv head) that gets rows
 * in this call, of K and of V, with c the scale before the call:
 *   c' = max(c, 2^e), e the least integer with max|x| <= 448 * 2^e over the
 *        finite entries x of those rows, clamped to [-64, 119];
 *   the rows' codes are x / c' rounded to nearest-even; magnitudes above 448
 *        (infinities) become 448, NaN stays NaN;
 *   if c' > c, the codes of the block's other rows become code * (c / c'),
 *        rounded the same way.
 * A row at offset 0 begins the block anew, as a sequence fills its blocks in
 * order: c counts as 0 then and the block's other rows are left as they were.
 * c = 0 likewise; any other c outside [2^-96, FLT_MAX] sets PKV_STATUS_BAD_SCALE and
 * counts as 0.  Tokens may come in any order; of several tokens with the same
 * slot the last one is stored.  The result does not depend on timing.
 *   workspace      device, >= pkv_kv_store_fp8_workspace_bytes(...) bytes,
 *                  16-byte aligned
 * Calls that store into the same block must not overlap on the GPU.
 */
PKV_API int pkv_kv_store_fp8(const void* k, const void* v, void* k_cache, void* v_cache,
                             float* k_scale, float* v_scale, const int32_t* slot_mapping,
                             int32_t num_tokens, void* workspace, size_t workspace_bytes,
                             pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * Bytes of device workspace pkv_paged_decode_fp8 needs (as
 * pkv_paged_decode_workspace_bytes; its chunks are longer).
 */
PKV_API size_t pkv_paged_decode_fp8_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                                    int32_t max_context_len,
                                                    pkv_cache_desc cache);

/*
 * paged_decode over an e4m3 cache: arguments and result as in
 * pkv_paged_decode, with K and V rows code * scale.  The keys of a block whose K or V scale cannot be
 * used are left out, as are those of a block id outside the pool.
 * V scales may differ by any factor within a sequence: every key counts in the softmax's sum.
 * In the sum of V rows a key's share (its weight times its V scale) is held to 2^-9 + 2^-11
 * of itself or to 2^-22 of the largest share among the keys attended together (2048 at most),
 * whichever is more: beside keys of the same weight and a V scale 2^13 larger, a small block's
 * values keep 9 bits, beside 2^20 two.
 */
PKV_API int pkv_paged_decode_fp8(const void* q, const void* k_cache, const void* v_cache,
                                 const float* k_scale, const float* v_scale,
                                 const int32_t* block_tables, int32_t max_blocks_per_seq,
                                 const int32_t* context_lens, int32_t batch,
                                 int32_t num_q_heads, int32_t max_context_len, float scale,
                                 void* out, void* workspace, size_t workspace_bytes,
                                 pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * paged_decode_fp8 split into a plan and a run, as pkv_paged_decode_plan and
 * pkv_paged_decode_run split pkv_paged_decode, under the same conditions.
 */
PKV_API int pkv_paged_decode_plan_fp8(const int32_t* context_lens, int32_t batch,
                                      int32_t num_q_heads, int32_t max_context_len,
                                      int32_t max_blocks_per_seq, void* workspace,
                                      size_t workspace_bytes, pkv_cache_desc cache,
                                      uint32_t* status, void* stream);
PKV_API int pkv_paged_decode_run_fp8(const void* q, const void* k_cache, const void* v_cache,
                                     const float* k_scale, const float* v_scale,
                                     const int32_t* block_tables, int32_t max_blocks_per_seq,
                                     const int32_t* context_lens, int32_t batch,
                                     int32_t num_q_heads, int32_t max_context_len, float scale,
                                     void* out, void* workspace, size_t workspace_bytes,
                                     pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * kv_store_fp8 then paged_decode_fp8, enqueued as one call; every argument is
 * checked before anything is enqueued.
 */
PKV_API size_t pkv_kv_store_paged_decode_fp8_workspace_bytes(int32_t num_tokens, int32_t batch,
                                                             int32_t num_q_heads,
                                                             int32_t max_context_len,
                                                             pkv_cache_desc cache);
PKV_API int pkv_kv_store_paged_decode_fp8(
    const void* k, const void* v, const int32_t* slot_mapping, int32_t num_tokens,
    const void* q, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
    const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
    int32_t batch, int32_t num_q_heads, int32_t max_context_len, float scale, void* out,
    void* workspace, size_t workspace_bytes, pkv_cache_desc cache, uint32_t* status,
    void* stream);

/*
 * Bytes of device workspace pkv_paged_prefill_varlen_fp8 needs (pure host
 * function): the tile schedule, partial results where few queries' keys are
 * split over several work items, and the prefixes' rows as bf16.  The latter are
 * sized for max_seqlen_k keys of every sequence, up to 4.1 GB; beyond that the
 * batch is attended in groups of sequences that share it (a single sequence may
 * need more).  The answer grows with batch, total_q and max_seqlen_k: a workspace
 * for the largest call serves the smaller ones.
 */
PKV_API size_t pkv_paged_prefill_fp8_workspace_bytes(int32_t batch, int32_t total_q,
                                                     int32_t num_q_heads, int32_t max_seqlen_k,
                                                     pkv_cache_desc cache);

/*
 * paged_prefill_varlen whose cached prefix lies in an e4m3 cache: arguments
 * and result as in pkv_paged_prefill_varlen, with prefix rows code * scale
 * (rounded to bf16, which is exact for power-of-two scales).  The chunk's own
 * keys are the bf16 rows of k / v.  A prefix row in a block id outside the pool
 * (PKV_STATUS_BAD_BLOCK_ID) or with a scale that cannot be used
 * (PKV_STATUS_BAD_SCALE) counts as zeros.  A sequence of more than max_seqlen_k keys
 * or more cached keys than its table holds sets PKV_STATUS_BAD_SEQLENS and is
 * skipped (its output rows are not written), as an inconsistent one is.
 */
PKV_API int pkv_paged_prefill_varlen_fp8(
    const void* q, const void* k, const void* v, const void* k_cache, const void* v_cache,
    const float* k_scale, const float* v_scale, const int32_t* cu_seqlens_q,
    const int32_t* cu_seqlens_k, int32_t batch, int32_t total_q, int32_t max_seqlen_q,
    int32_t max_seqlen_k, int32_t num_q_heads, const int32_t* block_tables,
    int32_t max_blocks_per_seq, float scale, void* out, void* workspace, size_t workspace_bytes,
    pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * ---- rules on a step's logits, ahead of pkv_sample -----------------------
 * (No counterpart on the pages, whose sampler takes the model's logits.)
 */
#define PKV_FP32 0
#define PKV_BF16 1
#define PKV_FP16 2

/* Device arrays; a NULL one (and what belongs to it) is not applied. */
typedef struct pkv_logit_rules {
    const int32_t* token_ids;            /* [batch, max_tokens]: prompt, then generated tokens  */
    const int32_t* prompt_lens;          /* [batch]: prompt tokens of each row; NULL: 0         */
    const int32_t* token_lens;           /* [batch]: all tokens of each row; NULL: max_tokens   */
    const float* repetition_penalties;   /* [batch], in [2^-100, 2^100]; NULL: 1                 */
    const float* presence_penalties;     /* [batch]; NULL: 0                                    */
    const float* frequency_penalties;    /* [batch]; NULL: 0                                    */
    const int32_t* bias_offsets;         /* [batch + 1]: row b has biases [off[b], off[b + 1])  */
    const int32_t* bias_token_ids;       /* [num_biases]                                        */
    const float* bias_values;            /* [num_biases]                                        */
    const uint32_t* allowed_mask;        /* [batch, ceil(vocab / 32)]: bit i % 32 of word i / 32 */
    int32_t max_tokens;
    int32_t num_biases;
} pkv_logit_rules;

/*
 * apply_logit_rules -- for entry i of row b, x = logits[b, i] in fp32, in this
 * order:
 *   repetition  if i occurs among the row's tokens: x = x > 0 ? x / r : x * r
 *               (x / r as x times the rounded 1 / r, one rounding more)
 *   frequency   x -= f * n, n the occurrences among the generated tokens (those
 *               behind the prompt)
 *   presence    x -= p if n > 0
 *   bias        x += the value of the row's last bias for token i
 *   mask        x = -inf where the token is not allowed
 *
 *   logits       device, [batch, vocab] of logits_type (PKV_FP32, PKV_BF16 or
 *                PKV_FP16), rows logits_stride entries apart
 *   out          device, [batch, vocab] fp32, contiguous.  May be logits itself
 *                (fp32, logits_stride == vocab): then entries that no rule changes
 *                are not written.  Any other overlap is PKV_ERR_UNSUPPORTED.
 * Token ids < 0 (padding) are skipped; one >= vocab sets PKV_STATUS_BAD_TOKEN_ID and
 * is skipped.  Inconsistent lengths or bias offsets set PKV_STATUS_BAD_SEQLENS
 * and that list of the row counts as empty.  A repetition penalty outside
 * [2^-100, 2^100] counts as 1, another penalty that is not finite as 0, and sets
 * PKV_STATUS_BAD_PENALTY.  A row whose mask allows no token becomes -inf
 * throughout and sets PKV_STATUS_NO_ALLOWED_TOKEN.
 */
PKV_API int pkv_apply_logit_rules(const void* logits, int32_t logits_type,
                                  int64_t logits_stride, int32_t batch, int32_t vocab,
                                  pkv_logit_rules rules, float* out, uint32_t* status,
                                  void* stream);

/*
 * ---- norms of q and k heads, and the rotation of their positions ----------
 * (No counterpart on the pages, whose attention takes rotated rows: the steps
 * between a layer's projections and its kv_store.)
 *
 * The first rotary_dim entries of a head are rotated in pairs: entries i and
 * i + rotary_dim / 2, or 2i and 2i + 1 where `interleaved` is not 0.  Pair i of
 * a token at position p turns by p * frequency[i] radians.  `turns` holds each
 * frequency as the fraction of a turn a position adds, in units of 2^-64
 * (pkv_rotary_turns), so that angles are exact to |p| * 2^-65 turns for any int32 p.
 */
typedef struct pkv_rotary {
    const uint64_t* turns;   /* device, [rotary_dim / 2]; NULL where rotary_dim is 0 */
    int32_t rotary_dim;      /* even, 0 (no rotation) .. head_dim */
    int32_t interleaved;
    float magnitude;         /* factor of the rotated entries */
} pkv_rotary;

/* How frequencies are stretched to positions beyond a model's training. */
#define PKV_ROPE_PLAIN  0    /* w_i = base^(-2i / rotary_dim)                              */
#define PKV_ROPE_LINEAR 1    /* w_i / factor                                               */
#define PKV_ROPE_NTK    2    /* base * factor^(rotary_dim / (rotary_dim - 2)) as the base   */
#define PKV_ROPE_YARN   3    /* w_i up to the pair that makes `high` turns within
                                original_max_position positions, w_i / factor from the one
                                that makes `low`, a ramp over the pairs between them;
                                magnitude 0.1 ln(factor) + 1                               */
#define PKV_ROPE_BANDS  4    /* by the turns w_i makes within original_max_position
                                positions: w_i from `high` on, w_i / factor up to `low`,
                                linear in the turns between them                           */
typedef struct pkv_rotary_scaling {
    int32_t kind;            /* PKV_ROPE_* */
    int32_t original_max_position;
    double factor;           /* >= 1 */
    double low, high;        /* turns: usually 1 and 32 (YARN), 1 and 4 (BANDS) */
} pkv_rotary_scaling;

/*
 * Host functions.  pkv_rotary_frequencies writes the rotary_dim / 2 frequencies
 * (radians a position) of a base (> 1) and a scaling to host memory, and the
 * magnitude that belongs to them.  pkv_rotary_turns turns any frequencies in
 * [0, 65536] into the units that pkv_rotary takes (to half a unit), in host memory;
 * the caller copies them to the device.
 */
PKV_API int pkv_rotary_frequencies(int32_t rotary_dim, double base, pkv_rotary_scaling scaling,
                                   double* frequencies, float* magnitude);
PKV_API int pkv_rotary_turns(const double* frequencies, int32_t count, uint64_t* turns);

/*
 * qk_norm_rope -- RMS norm and rotation of every q and k head: for a head x,
 *   y = x * weight / sqrt(mean(x^2) + eps)   (y = x where the weights are NULL),
 *   then y's first rotary_dim entries rotated by its token's position, pairs
 *   (a, b) -> magnitude * (a cos - b sin, b cos + a sin).
 * Computed in fp32 and rounded once to the rows' type; squares beyond fp32 do no
 * harm (such a head is scaled by a power of two first).
 *
 *   q, k         device, [num_tokens, heads, head_dim] of `type` (PKV_FP32, PKV_BF16
 *                or PKV_FP16), tokens q_stride / k_stride elements apart (a packed
 *                projection's rows)
 *   q_weight, k_weight  device, [head_dim] of weight_type, or NULL
 *   positions    device, [num_tokens] int32, any value
 *   q_out, k_out device, as q and k, with strides of their own.  Either may be its own
 *                input (same stride); any other overlap is PKV_ERR_UNSUPPORTED.
 * head_dim a multiple of 8, at most 256; rows 16-byte aligned.  A norm or a
 * rotation is needed (PKV_ERR_BAD_DIMENSION otherwise).  Strides are not read when
 * num_tokens is 1.
 */
PKV_API int pkv_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             int32_t type, const void* q_weight, const void* k_weight,
                             int32_t weight_type, float eps, const int32_t* positions,
                             pkv_rotary rotary, int32_t num_tokens, int32_t num_q_heads,
                             int32_t num_kv_heads, int32_t head_dim, void* q_out,
                             int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                             void* stream);

/*
 * qk_norm_rope of bf16 rows and kv_store in one pass: q rows to q_out, k rows
 * normed and rotated to their slots of k_cache (and to k_out unless it is
 * NULL, e.g. for pkv_paged_prefill_varlen), v rows [num_tokens, num_kv_heads,
 * head_dim], v_stride elements apart, to their slots of v_cache as they are.
 * slot_mapping as in pkv_kv_store, but of tokens with the same slot the last
 * one's rows are stored; a token without a slot still gets its q_out and k_out
 * rows.  The caches must not overlap the other tensors.
 */
PKV_API int pkv_qk_norm_rope_kv_store(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const void* q_weight, const void* k_weight, int32_t weight_type, float eps,
    const int32_t* positions, pkv_rotary rotary, const int32_t* slot_mapping, int32_t num_tokens,
    int32_t num_q_heads, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
    void* k_cache, void* v_cache, pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * ---- decode attention over shared prefixes --------------------------------
 * (No counterpart on the pages, whose prefix cache lets sequences share blocks;
 * here their attention shares the work on them too.)
 *
 * Bytes of device workspace the calls below need (a pure host function).  As
 * with pkv_paged_decode_workspace_bytes, a workspace shared by several batch
 * sizes must be as large as the largest of their answers.  With 32 q and 8 kv heads
 * of 128 and contexts of 1500: 4 MB for 8 sequences, 21 for 64, 69 for 256; at most
 * 95 for 256 of any length.
 */
PKV_API size_t pkv_paged_decode_shared_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                                       int32_t max_context_len,
                                                       pkv_cache_desc cache);

/*
 * paged_decode for sequences in groups whose first keys are the same: arguments
 * and result as in pkv_paged_decode, and
 *   group_offsets device, [num_groups + 1] int32, increasing, within [0, batch]:
 *                 group g is the sequences group_offsets[g] .. group_offsets[g+1] - 1.
 *                 Sequences outside every group attend by themselves.
 *   prefix_lens   device, [num_groups] int32: the first prefix_lens[g] keys of every
 *                 sequence of group g (of its context_lens[b] in all) are those that
 *                 any one of its block-table rows names.  Loaded once for every 128
 *                 rows (query heads of a kv head, times sequences) of the group.
 * num_groups 0 takes NULL for both.  scale must be positive and finite.
 * A context length of 0 gives zeros.  One below its group's prefix, or out of
 * range as in pkv_paged_decode, sets PKV_STATUS_BAD_CONTEXT_LEN and gives zeros.
 * Offsets that decrease or leave the batch set PKV_STATUS_BAD_SEQLENS and no group
 * is used; a prefix < 0 or longer than max_context_len or the block table sets it
 * and counts as 0.  Keys in a block id outside the pool are left out.  A query
 * row whose scores are NaN or, times log2 e, pass 32 bits gives NaN.
 * num_blocks*block_size must be below 2^31 and max_context_len at most 2^30
 * (PKV_ERR_UNSUPPORTED; the workspace's size is 0 then).
 * Its plan takes 5 us where pkv_paged_decode's takes 2: with 32 q and 8 kv heads of
 * 128 and up to 1500 own keys the whole call is as fast as pkv_paged_decode at
 * about 100 common keys of 256 sequences, 200 of 64, 500 of 8, 2500 of two, and
 * faster from there on (64 and 1024: 52 us for 81); a run alone at 64, 100, 130 and
 * 2000.
 */
PKV_API int pkv_paged_decode_shared(const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, int32_t max_blocks_per_seq,
                                    const int32_t* context_lens, const int32_t* group_offsets,
                                    const int32_t* prefix_lens, int32_t num_groups, int32_t batch,
                                    int32_t num_q_heads, int32_t max_context_len, float scale,
                                    void* out, void* workspace, size_t workspace_bytes,
                                    pkv_cache_desc cache, uint32_t* status, void* stream);

/*
 * paged_decode_shared split into a plan (of the lengths alone, once a step) and a
 * run (once a layer), as pkv_paged_decode_plan and pkv_paged_decode_run split
 * pkv_paged_decode, under the same conditions.
 */
PKV_API int pkv_paged_decode_plan_shared(const int32_t* context_lens, const int32_t* group_offsets,
                                         const int32_t* prefix_lens, int32_t num_groups,
                                         int32_t batch, int32_t num_q_heads,
                                         int32_t max_context_len, int32_t max_blocks_per_seq,
                                         void* workspace, size_t workspace_bytes,
                                         pkv_cache_desc cache, uint32_t* status, void* stream);
PKV_API int pkv_paged_decode_run_shared(const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                                        int32_t batch, int32_t num_q_heads,
                                        int32_t max_context_len, float scale, void* out,
                                        void* workspace, size_t workspace_bytes,
                                        pkv_cache_desc cache, uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */
