// Declarations shared by the two paged_decode split kernels (paged_decode.cu:
// loads straight into registers, any block size; paged_decode_tma.cu: a TMA
// producer warp feeding a shared-memory ring, block sizes that are multiples
// of 64) and by the plan and combine kernels they share.
#pragma once

#include "common.cuh"

namespace pkv {

constexpr int kMaxGroup = 8;         // q heads per unit (mma rows 0..7)

struct DecodeArgs {
    const __nv_bfloat16* q;
    const __nv_bfloat16* kc;
    const __nv_bfloat16* vc;
    const int32_t* bt;
    const int32_t* ctx;
    __nv_bfloat16* out;
    int32_t* chunk_prefix;           // [B+1] exclusive prefix of chunk counts
    int4* chunk_info;                // [cap]: (sequence, first key, end key, chunks of it)
    float2* part_ml;                 // [cap * Hq]: (max, sum) in base 2 (e4m3 cache: max halved)
    float* part_o;                   // [cap * Hq * D]
    int32_t B, Hq, Hkv, G, n_hg, MB, NB, bs, max_ctx, chunk_keys, cap;
    float scale_log2;
    uint32_t* status;
    // A varlen batch (mixed prefill and decode): when cu_q is set, sequence b
    // is a decode row only if cu_q[b+1] - cu_q[b] == 1; its q and out row is
    // cu_q[b] and its context cu_k[b+1] - cu_k[b].  Other sequences get no
    // chunks and their out rows are left alone.
    const int32_t* cu_q;
    const int32_t* cu_k;
    int32_t total_q;                 // rows of q / out (varlen batch only)
    int32_t b0;                      // first sequence of a combine launch
    uint32_t wait_polls;             // polls of a bounded mbarrier wait
    // No plan in the workspace: the kernels take the schedule of a batch of at
    // most kMaxInline sequences from `ctx` themselves (WarpPlan).
    int32_t inline_plan;
};

// The chunk schedule of at most kMaxInline sequences, held by a warp: lane l has
// sequence 32 i + l's length, chunks and the chunks up to and with it.  What the
// plan kernel writes for any number, without its launch.
constexpr int kInlinePerLane = 4, kMaxInline = 32 * kInlinePerLane;

struct WarpPlan {
    int32_t len[kInlinePerLane], n[kInlinePerLane], incl[kInlinePerLane];
    int32_t batch, sum;              // chunks of all
    bool bad;                        // one of this lane's lengths is out of range (no chunks)
    __device__ __forceinline__ explicit WarpPlan(const DecodeArgs& a) {
        const int lane = threadIdx.x & 31;
        bad = false;
        batch = a.B;
#pragma unroll
        for (int i = 0; i < kInlinePerLane; ++i)
            len[i] = 32 * i + lane < batch ? a.ctx[32 * i + lane] : 0;
        int32_t before = 0;
#pragma unroll
        for (int i = 0; i < kInlinePerLane; ++i) {
            n[i] = 0;
            incl[i] = before;
            if (i > 0 && 32 * i >= batch) continue;
            const bool out = len[i] < 0 || len[i] > (int64_t)a.MB * a.bs || len[i] > a.max_ctx;
            bad |= out;
            int32_t x = n[i] = out ? 0 : (len[i] + a.chunk_keys - 1) / a.chunk_keys;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += y;
            }
            incl[i] += x;
            before = __shfl_sync(0xffffffffu, incl[i], 31);
        }
        sum = before;
    }
    __device__ __forceinline__ int32_t total() const { return sum; }
    // a sequence's value (b alike in every lane)
    __device__ __forceinline__ static int32_t get(const int32_t (&x)[kInlinePerLane], int32_t b) {
        if (b < 32) return __shfl_sync(0xffffffffu, x[0], b);
        int32_t mine = x[1];
#pragma unroll
        for (int i = 2; i < kInlinePerLane; ++i)
            if (b >= 32 * i) mine = x[i];
        return __shfl_sync(0xffffffffu, mine, b & 31);
    }
    // (first chunk, chunks) of sequence b
    __device__ __forceinline__ int2 of(int32_t b) const {
        const int32_t nb = get(n, b);
        return make_int2(get(incl, b) - nb, nb);
    }
    // (sequence, first key, end key, chunks of the sequence) of chunk sc < total()
    __device__ __forceinline__ int4 record(int32_t sc, int32_t chunk_keys) const {
        int32_t b = __popc(__ballot_sync(0xffffffffu, incl[0] <= sc));
        if (batch > 32) {
#pragma unroll
            for (int i = 1; i < kInlinePerLane; ++i)
                b += __popc(__ballot_sync(0xffffffffu, incl[i] <= sc));
        }
        const int2 f = of(b);
        const int32_t i = sc - f.x;
        return make_int4(b, i * chunk_keys, min(get(len, b), (i + 1) * chunk_keys), f.y);
    }
};

// q / out row of sequence b
__device__ __forceinline__ int64_t row_of(const DecodeArgs& a, int32_t b) {
    return a.cu_q != nullptr ? (int64_t)a.cu_q[b] : (int64_t)b;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// pack (lo = element e of a, hi = element e of b), e in 0..7 of a 16-byte chunk
__device__ __forceinline__ uint32_t pair(const uint4& a, const uint4& b, int e) {
    return __byte_perm(word(a, e >> 1), word(b, e >> 1), (e & 1) ? 0x7632 : 0x5410);
}

__device__ __forceinline__ void allow_dependent_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_predecessor() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace pkv

// The TMA split kernel (paged_decode_tma.cu).  `supported` returns PKV_OK when
// the shapes are its own; `launch` enqueues the split kernel only, as a
// programmatic dependent of the plan kernel.
int pkv_decode_tma_supported(const pkv::DecodeArgs& a, int head_dim);
int pkv_launch_decode_tma(pkv::DecodeArgs& a, int head_dim, cudaStream_t s);

// Pieces of pkv_paged_decode (paged_decode.cu) that the decode over an e4m3
// cache shares, with a chunk length of its own: the workspace, the argument checks
// (the cache pointers are checked and stored untyped), the plan kernel, and its
// combine kernel as a programmatic dependent of the split kernel before it.
size_t pkv_decode_workspace(int32_t batch, int32_t num_q_heads, int32_t max_context_len,
                            const pkv_cache_desc& cache, int32_t chunk_keys);
int pkv_decode_make_plan_args(const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
                              int32_t max_context_len, int32_t max_blocks_per_seq,
                              void* workspace, size_t workspace_bytes,
                              const pkv_cache_desc& cache, uint32_t* status, pkv::DecodeArgs& a,
                              int32_t chunk_keys);
int pkv_decode_make_args(const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                         const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
                         int32_t max_context_len, float scale, void* out, void* workspace,
                         size_t workspace_bytes, const pkv_cache_desc& cache, uint32_t* status,
                         pkv::DecodeArgs& a, int32_t chunk_keys);
int pkv_launch_decode_plan(const pkv::DecodeArgs& a, cudaStream_t s);
int pkv_launch_decode_combine(const pkv::DecodeArgs& a, int head_dim, cudaStream_t s);
