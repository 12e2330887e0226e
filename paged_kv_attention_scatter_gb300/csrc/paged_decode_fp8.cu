// paged_decode_fp8: split-KV decode attention over an e4m3 cache with one
// scale for each (cache block, kv head).
//
// What it computes: as paged_decode, with key and value rows
// K_j = ks * K8_j and V_j = vs * V8_j, where ks, vs are the scales of key j's
// block and kv head:
//   x_j = scale * ks_j * (q . K8_j),  out = sum_j softmax(x)_j * vs_j * V8_j.
//
// The scales never touch a code: ks multiplies the score, and vs rides in the
// exponent.  With y_j = x_j + log2 vs_j (base 2) and M the running maximum of y,
//   p_j = 2^(y_j - M) = 2^(x_j - M) vs_j,
//   O = sum p_j V8_j,   L = sum p_j / vs_j,   out = O / L,
// so p is at most 1 whatever the scales, one exponential serves both sums, and a
// (M, L, O) triple merges across chunks as in the bf16 decode, with that decode's plan
// kernel.  The scales span 2^224, more than fp32's exponent does below 1: a key of a
// small scale beside one of a large scale may have no p left, but its share of L has
// to count.  So p is squared up from g = 2^((y - M) / 2), which is normal down to
// y - M = -252, and L sums (g / sqrt(vs))^2; where M rises or triples merge, L is
// scaled by half the power twice.  O loses nothing that shows: a key's part of it is
// held to 2^-9 of itself or 2^-22 of the largest p (paged_decode_fp8_tc.cu), that is of
// the largest product of a weight and a V scale among the at most 2048 keys of a unit.
// The split kernel is in paged_decode_fp8_tc.cu; this file has the entry points.
#include "fp8_common.cuh"

namespace {

using pkv::Fp8DecodeArgs;
using pkv::kMaxGroup;

// Keys per work unit, from the sizes alone (152 SMs, a GB300's, are written down because
// the workspace's size follows): the multiple of 128 (a stage of
// head_dim 128) nearest to the length that gives about two units per SM for a
// typical context of half the stated maximum, within 128..1024, and 2048 (a lane of
// the producer has one of a unit's 64-key boxes) where a SM has sixteen such units or
// where a stage of head_dim 64 has eight heads' softmax.  A unit's end
// -- its last stage's P V waited for, the two softmax groups' shares merged --
// costs about a stage, so units are longer than the bf16 decode's, whose rule
// aims at sixteen a SM (measured, us: 64 sequences of 16/8 heads and 512..4096
// keys 61 at 256, 56 at 512, 55 at 1024; 8 of 32/8 and 4000..8192 43 at 128, 27 at
// 512, 25 at 1024; 2 of 30000..32768 68, 34, 32; and at 1024 and 2048: 64 of 16/8 as
// above 55, 60; 96 of 64/8 and 128..32768 198, 196; head_dim 64, 64 of 64/8 and
// 512..4096 50, 48, in blocks of 16 67, 62; of 16/8 36, 38).
int32_t choose_chunk_keys(int32_t batch, int32_t num_q_heads, int32_t max_ctx,
                          const pkv_cache_desc& c) {
    const int32_t hkv = c.num_kv_heads > 0 ? c.num_kv_heads : 1;
    const int32_t n_hg = (num_q_heads / hkv + kMaxGroup - 1) / kMaxGroup;
    const double keys = (double)max_ctx / 2.0 * batch * hkv * n_hg / (2.0 * 152);
    const double chunk = keys / 128.0 + 0.5;
    // short contexts: one unit a sequence and head, so that nothing is left to combine
    if (max_ctx <= 512) return max_ctx <= 128 ? 128 : (max_ctx + 127) / 128 * 128;
    if (chunk < 1.0) return 128;
    if (chunk >= 128.0 || (chunk >= 16.0 && c.head_dim == 64 && num_q_heads / hkv > 4)) return 2048;
    return chunk >= 8.0 ? 1024 : (int32_t)chunk * 128;
}

// Plan, split, combine.  A batch of at most 128 sequences needs no plan kernel (nor
// has one if a plan is in the workspace), and one of single chunks no combine: a
// small call's time is mostly its launches' (48 sequences of 32/8 heads and 1..8192
// keys, block size 16: 82 us with a plan kernel, 77 without; a lane has up to four
// sequences of the schedule).
int launch_decode(Fp8DecodeArgs& fa, int head_dim, bool plan, cudaStream_t s) {
    int rc = PKV_OK;
    fa.d.inline_plan = plan && fa.d.B <= pkv::kMaxInline;
    fa.no_combine = fa.d.max_ctx <= fa.d.chunk_keys;
    if (plan && !fa.d.inline_plan) rc = pkv_launch_decode_plan(fa.d, s);
    if (rc != PKV_OK) return rc;
    rc = pkv_launch_decode_fp8(fa, head_dim, s);
    if (rc != PKV_OK || fa.no_combine) return rc;
    return pkv_launch_decode_combine(fa.d, head_dim, s);
}

int make_args(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
              const float* v_scale, const int32_t* block_tables, int32_t max_blocks_per_seq,
              const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
              int32_t max_context_len, float scale, void* out, void* workspace,
              size_t workspace_bytes, const pkv_cache_desc& cache, uint32_t* status,
              Fp8DecodeArgs& fa) {
    const int rc = pkv_decode_make_args(q, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                        context_lens, batch, num_q_heads, max_context_len, scale,
                                        out, workspace, workspace_bytes, cache, status, fa.d,
                                        choose_chunk_keys(batch, num_q_heads, max_context_len,
                                                          cache));
    if (rc != PKV_OK) return rc;
    if (!k_scale || !v_scale) return PKV_ERR_NULL_POINTER;
    if (((uintptr_t)k_scale | (uintptr_t)v_scale) & 3) return PKV_ERR_MISALIGNED;
    if (cache.block_size > pkv::kFp8MaxBlockSize) return PKV_ERR_BAD_DIMENSION;
    if ((int64_t)cache.num_blocks * cache.block_size >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;
    fa.kc = (const uint8_t*)k_cache;
    fa.vc = (const uint8_t*)v_cache;
    fa.ks = k_scale;
    fa.vs = v_scale;
    return PKV_OK;
}

}  // namespace

extern "C" size_t pkv_paged_decode_fp8_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                                       int32_t max_context_len,
                                                       pkv_cache_desc cache) {
    if (batch < 0 || num_q_heads <= 0 || max_context_len < 0 || cache.num_kv_heads <= 0 ||
        cache.head_dim <= 0)
        return 0;
    return pkv_decode_workspace(batch, num_q_heads, max_context_len, cache,
                                choose_chunk_keys(batch, num_q_heads, max_context_len, cache));
}

extern "C" int pkv_paged_decode_plan_fp8(const int32_t* context_lens, int32_t batch,
                                         int32_t num_q_heads, int32_t max_context_len,
                                         int32_t max_blocks_per_seq, void* workspace,
                                         size_t workspace_bytes, pkv_cache_desc cache,
                                         uint32_t* status, void* stream) {
    if (batch == 0 && max_context_len >= 0 && num_q_heads > 0) return PKV_OK;
    pkv::DecodeArgs a{};
    const int rc = pkv_decode_make_plan_args(
        context_lens, batch, num_q_heads, max_context_len, max_blocks_per_seq, workspace,
        workspace_bytes, cache, status, a,
        choose_chunk_keys(batch, num_q_heads, max_context_len, cache));
    return rc != PKV_OK ? rc : pkv_launch_decode_plan(a, (cudaStream_t)stream);
}

extern "C" int pkv_paged_decode_fp8(const void* q, const void* k_cache, const void* v_cache,
                                    const float* k_scale, const float* v_scale,
                                    const int32_t* block_tables, int32_t max_blocks_per_seq,
                                    const int32_t* context_lens, int32_t batch,
                                    int32_t num_q_heads, int32_t max_context_len, float scale,
                                    void* out, void* workspace, size_t workspace_bytes,
                                    pkv_cache_desc cache, uint32_t* status, void* stream) {
    if (batch == 0 && max_context_len >= 0 && num_q_heads > 0) return PKV_OK;
    Fp8DecodeArgs fa{};
    const int rc = make_args(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                             max_blocks_per_seq, context_lens, batch, num_q_heads,
                             max_context_len, scale, out, workspace, workspace_bytes, cache,
                             status, fa);
    return rc != PKV_OK ? rc : launch_decode(fa, cache.head_dim, true, (cudaStream_t)stream);
}

extern "C" int pkv_paged_decode_run_fp8(const void* q, const void* k_cache, const void* v_cache,
                                        const float* k_scale, const float* v_scale,
                                        const int32_t* block_tables, int32_t max_blocks_per_seq,
                                        const int32_t* context_lens, int32_t batch,
                                        int32_t num_q_heads, int32_t max_context_len,
                                        float scale, void* out, void* workspace,
                                        size_t workspace_bytes, pkv_cache_desc cache,
                                        uint32_t* status, void* stream) {
    if (batch == 0 && max_context_len >= 0 && num_q_heads > 0) return PKV_OK;
    Fp8DecodeArgs fa{};
    const int rc = make_args(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                             max_blocks_per_seq, context_lens, batch, num_q_heads,
                             max_context_len, scale, out, workspace, workspace_bytes, cache,
                             status, fa);
    return rc != PKV_OK ? rc : launch_decode(fa, cache.head_dim, false, (cudaStream_t)stream);
}

namespace {

// The store's list of runs lies behind the decode's workspace.
size_t store_at(int32_t batch, int32_t num_q_heads, int32_t max_context_len,
                const pkv_cache_desc& cache) {
    return (pkv_paged_decode_fp8_workspace_bytes(batch, num_q_heads, max_context_len, cache) +
            255) &
           ~(size_t)255;
}

}  // namespace

extern "C" size_t pkv_kv_store_paged_decode_fp8_workspace_bytes(
        int32_t num_tokens, int32_t batch, int32_t num_q_heads, int32_t max_context_len,
        pkv_cache_desc cache) {
    if (num_tokens < 0 || batch < 0 || num_q_heads <= 0 || max_context_len < 0 ||
        cache.num_blocks <= 0 || cache.num_kv_heads <= 0 || cache.head_dim <= 0)
        return 0;
    return store_at(batch, num_q_heads, max_context_len, cache) +
           pkv_kv_store_fp8_workspace_bytes(num_tokens, cache);
}

extern "C" int pkv_kv_store_paged_decode_fp8(
        const void* k, const void* v, const int32_t* slot_mapping, int32_t num_tokens,
        const void* q, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
        const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
        int32_t batch, int32_t num_q_heads, int32_t max_context_len, float scale, void* out,
        void* workspace, size_t workspace_bytes, pkv_cache_desc cache, uint32_t* status,
        void* stream) {
    const bool decode = !(batch == 0 && max_context_len >= 0 && num_q_heads > 0);
    Fp8DecodeArgs fa{};
    size_t at = 0;
    if (decode) {
        const int rc = make_args(q, k_cache, v_cache, k_scale, v_scale, block_tables,
                                 max_blocks_per_seq, context_lens, batch, num_q_heads,
                                 max_context_len, scale, out, workspace, workspace_bytes, cache,
                                 status, fa);
        if (rc != PKV_OK) return rc;                          // nothing enqueued
        at = store_at(batch, num_q_heads, max_context_len, cache);
    }
    const size_t left = workspace_bytes > at ? workspace_bytes - at : 0;
    const Fp8StoreCall st{k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, num_tokens,
                          workspace ? (char*)workspace + at : nullptr, left, cache, status};
    int rc = pkv_kv_store_fp8_check(st);
    if (rc != PKV_OK) return rc;                              // nothing enqueued
    cudaStream_t s = (cudaStream_t)stream;
    rc = pkv_kv_store_fp8_launch(st, s);
    if (rc != PKV_OK || !decode) return rc;
    return launch_decode(fa, cache.head_dim, true, s);
}
