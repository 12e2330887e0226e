// paged_decode_fp8: split-KV decode attention over an e4m3 cache with one
// scale for each (cache block, kv head).
//
// What it computes: as paged_decode, with key and value rows
// K_j = ks * K8_j and V_j = vs * V8_j, where ks, vs are the scales of key j's
// block and kv head:
//   x_j = scale * ks_j * (q . K8_j),  out = sum_j softmax(x)_j * vs_j * V8_j.
//
// The arithmetic.  Codes become f16, which holds every e4m3 value exactly, and
// both products run on the tensor pipe in f16 with fp32 accumulation.  q is
// bf16, whose range f16 lacks: each q row is multiplied by a power of two that
// brings its largest entry to [2^14, 2^15), which loses nothing down to 2^-29 of
// that entry, and the power is taken out of x in fp32.  The scales never touch
// a code: ks multiplies the score, and vs rides in the exponent.  With
// y_j = x_j + log2 vs_j (base 2) and M the running maximum of y,
//   p_j = 2^(y_j - M) = 2^(x_j - M) vs_j,
//   O = sum p_j V8_j,   L = sum p_j / vs_j,   out = O / L,
// so p is at most 1 whatever the scales, one exponential serves both sums, and a
// (M, L, O) triple merges across chunks as in the bf16 decode: the plan and
// the combine kernel are that decode's.  p is rounded to f16 (2^-11) for the
// product; L takes it unrounded.
//
// This file has the entry points and a split kernel for any block size; the
// one for block sizes that are multiples of 64 is in paged_decode_fp8_tma.cu.
#include "fp8_common.cuh"
#include <stdlib.h>

namespace {

using pkv::Fp8DecodeArgs;
using pkv::kMaxGroup;
using pkv::word;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;            // keys per warp step

// Loads straight into mma fragments, 16 keys a warp step (see paged_decode.cu
// for the fragment layouts; a 16-byte load holds 16 codes here).
//   S = Q K^T: lane (g, t) loads chunks t, t + 4 of key rows g and 8 + g; a
//   word of four codes is one k-step's pair of B registers, and q is laid out
//   to match.
//   O^T = V^T P^T: lane (g, t) loads chunk g (16 codes; 8 for head_dim 64) of
//   the rows of keys 2t, 2t + 1, 2t + 8, 2t + 9.  A byte permute of two rows
//   gives codes (e of row a, e of row b, e + 1 of a, e + 1 of b), whose
//   conversion is two A registers, for head_dim rows e and e + 1.
template <int D>
__global__ void __launch_bounds__(kThreads) decode_fp8_split_kernel(Fp8DecodeArgs fa) {
    const pkv::DecodeArgs& a = fa.d;
    constexpr int NC = D / 64;       // 16-byte chunks per lane of a K row
    constexpr int KK = D / 16;       // k-steps of S = Q K^T
    constexpr int MT = D / 16;       // m-tiles of O^T
    constexpr int VE = D / 8;        // codes per lane of a V row
    __shared__ float sm_m[kWarps][kMaxGroup];
    __shared__ float sm_l[kWarps][kMaxGroup];
    __shared__ float sm_o[kWarps][kMaxGroup][D];

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    pkv::wait_for_predecessor();             // the plan kernel's chunk records
    pkv::allow_dependent_launch();
    const int units_per_sc = a.Hkv * a.n_hg;
    const int64_t units = (int64_t)a.chunk_prefix[a.B] * units_per_sc;
    const int64_t row_codes = (int64_t)a.Hkv * D;

    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int32_t sc = (int32_t)(u / units_per_sc);
        const int32_t rem = (int32_t)(u - (int64_t)sc * units_per_sc);
        const int32_t kvh = rem / a.n_hg, hg = rem - kvh * a.n_hg;
        const int4 info = a.chunk_info[sc];
        const int32_t b = info.x, key0 = info.y, key_end = info.z, nch = info.w;
        const int32_t h0 = kvh * a.G + hg * kMaxGroup;
        const int32_t nh = min(kMaxGroup, a.G - hg * kMaxGroup);
        const int32_t* bt_row = a.bt + (int64_t)b * a.MB;
        const uint8_t* kbase = fa.kc + (int64_t)kvh * D;
        const uint8_t* vbase = fa.vc + (int64_t)kvh * D;

        uint32_t qa[KK][2];
        const float q_pow = pkv::load_q_f16<D>(
            a.q + ((int64_t)b * a.Hq + h0 + g) * D, g < nh, t, qa);
        const float x_scale = a.scale_log2 * q_pow;

        float o[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        float m_run = -INFINITY, l_run = 0.f;
        uint32_t bad = 0;

        for (int32_t step = key0 + warp * kStep; step < key_end; step += kWarps * kStep) {
            // lane l resolves key step + (l & 15): its block, row and scales
            const int32_t key = step + (lane & 15);
            int64_t row = -1;                // first code of the key's row, -1: masked
            float ks = 0.f, vs = 1.f;
            if (key < key_end) {
                const int32_t blk = bt_row[key / a.bs];
                if ((unsigned)blk < (unsigned)a.NB) {
                    const int64_t at = (int64_t)blk * a.Hkv + kvh;
                    const float k1 = __ldg(fa.ks + at), v1 = __ldg(fa.vs + at);
                    if (pkv::scale_ok(k1) && pkv::scale_ok(v1)) {
                        row = ((int64_t)blk * a.bs + key % a.bs) * row_codes;
                        ks = k1;
                        vs = v1;
                    } else {
                        bad |= PKV_STATUS_BAD_SCALE;
                    }
                } else {
                    bad |= PKV_STATUS_BAD_BLOCK_ID;
                }
            }
            const float lv = __log2f(vs), iv = __frcp_rn(vs);
            uint4 kr[2][NC];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t rr = __shfl_sync(0xffffffffu, row, r * 8 + g);
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    kr[r][i] = rr >= 0 ? pkv::ld_stream16(kbase + rr + (i * 4 + t) * 16)
                                       : make_uint4(0, 0, 0, 0);
            }
            uint32_t vr[4][VE / 4];
            bool valid[4];
            float kf[4], lf[4], vf[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int src = 2 * t + (r & 1) + 8 * (r >> 1);
                const int64_t rr = __shfl_sync(0xffffffffu, row, src);
                kf[r] = __shfl_sync(0xffffffffu, ks, src) * x_scale;
                lf[r] = __shfl_sync(0xffffffffu, lv, src);
                vf[r] = __shfl_sync(0xffffffffu, iv, src);
                valid[r] = rr >= 0;
#pragma unroll
                for (int c = 0; c < VE / 4; ++c) vr[r][c] = 0;
                if (valid[r]) {
                    if constexpr (VE == 16) {
                        const uint4 w = pkv::ld_stream16(vbase + rr + g * 16);
                        vr[r][0] = w.x;
                        vr[r][1] = w.y;
                        vr[r][2] = w.z;
                        vr[r][3] = w.w;
                    } else {
                        const uint2 w = __ldg(reinterpret_cast<const uint2*>(vbase + rr + g * 8));
                        vr[r][0] = w.x;
                        vr[r][1] = w.y;
                    }
                }
            }
            // ---- S = Q K^T for two 8-key tiles ----
            float s[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) {
                    uint32_t b0, b1;
                    pkv::e4m3x4_to_f16x4(word(kr[nt][kk >> 2], kk & 3), b0, b1);
                    pkv::mma_f16_16816(s[nt], qa[kk][0], 0u, qa[kk][1], 0u, b0, b1);
                }
            }
            // ---- online softmax (base 2) over keys 2t, 2t+1, 8+2t, 9+2t ----
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = valid[j] ? fmaf(s[j >> 1][j & 1], kf[j], lf[j]) : -INFINITY;
            float mx = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m_new = fmaxf(m_run, mx);
            const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
            const float alpha = (m_run == -INFINITY) ? 0.f : pkv::fast_exp2(m_run - m_use);
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = pkv::fast_exp2(y[j] - m_use);
            l_run = l_run * alpha + fmaf(p[0], vf[0], p[1] * vf[1]) +
                    fmaf(p[2], vf[2], p[3] * vf[3]);
            m_run = m_new;
            const float alpha_a = __shfl_sync(0xffffffffu, alpha, (2 * t) * 4);
            const float alpha_b = __shfl_sync(0xffffffffu, alpha, (2 * t + 1) * 4);
            const uint32_t b0 = pkv::pack_f16(p[0], p[1]);
            const uint32_t b1 = pkv::pack_f16(p[2], p[3]);
            // ---- O^T = V^T P^T: m-tile mt holds head_dim rows VE*g + 2mt, 2mt + 1 ----
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                o[mt][0] *= alpha_a; o[mt][1] *= alpha_b;
                o[mt][2] *= alpha_a; o[mt][3] *= alpha_b;
                uint32_t a0, a1, a2, a3;
                const uint32_t sel = (mt & 1) ? 0x7362 : 0x5140;
                pkv::e4m3x4_to_f16x4(__byte_perm(vr[0][mt >> 1], vr[1][mt >> 1], sel), a0, a1);
                pkv::e4m3x4_to_f16x4(__byte_perm(vr[2][mt >> 1], vr[3][mt >> 1], sel), a2, a3);
                pkv::mma_f16_16816(o[mt], a0, a1, a2, a3, b0, b1);
            }
        }
        if (bad) pkv::report(a.status, bad);

        // ---- per-warp results to shared memory ----
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
        l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
        if (t == 0) {
            sm_m[warp][g] = m_run;
            sm_l[warp][g] = l_run;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int d = VE * g + 2 * mt;
            *reinterpret_cast<float2*>(&sm_o[warp][2 * t][d]) = make_float2(o[mt][0], o[mt][2]);
            *reinterpret_cast<float2*>(&sm_o[warp][2 * t + 1][d]) =
                make_float2(o[mt][1], o[mt][3]);
        }
        __syncthreads();
        // ---- merge the 4 warps: thread -> (head, d) ----
        for (int idx = threadIdx.x; idx < nh * D; idx += kThreads) {
            const int h = idx / D, d = idx - h * D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][h]);
            float L = 0.f, O = 0.f;
            if (M != -INFINITY) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float mw = sm_m[w][h];
                    if (mw == -INFINITY) continue;
                    const float f = pkv::fast_exp2(mw - M);
                    L += sm_l[w][h] * f;
                    O += sm_o[w][h][d] * f;
                }
            }
            const int64_t qh = (int64_t)b * a.Hq + h0 + h;
            if (nch == 1) {
                a.out[qh * D + d] = __float2bfloat16_rn(L > 0.f ? O / L : 0.f);
            } else {
                const int64_t slot = (int64_t)sc * a.Hq + h0 + h;
                a.part_o[slot * D + d] = O;
                if (d == 0) a.part_ml[slot] = make_float2(M, L);
            }
        }
        __syncthreads();
    }
}

template <int D>
int launch_split(const Fp8DecodeArgs& fa, cudaStream_t s) {
    static std::atomic<int> resident[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    int per_sm = resident[dev].load(std::memory_order_relaxed);
    if (per_sm <= 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                &per_sm, (const void*)decode_fp8_split_kernel<D>, kThreads, 0) != cudaSuccess ||
            per_sm < 1)
            per_sm = 1;
        resident[dev].store(per_sm, std::memory_order_relaxed);
    }
    const pkv::DecodeArgs& a = fa.d;
    const int64_t upper = (int64_t)a.cap * a.Hkv * a.n_hg;
    int64_t grid = (int64_t)pkv_num_sms() * per_sm;
    if (grid > upper) grid = upper;
    if (grid < 1) grid = 1;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_fp8_split_kernel<D>, fa) == cudaSuccess
               ? PKV_OK : PKV_ERR_CUDA;
}

// Plan (unless a plan is in the workspace), split, combine.
int launch_decode(Fp8DecodeArgs& fa, int head_dim, bool plan, cudaStream_t s) {
    int rc = plan ? pkv_launch_decode_plan(fa.d, s) : PKV_OK;
    if (rc != PKV_OK) return rc;
    if (getenv("PKV_OLD") == nullptr)
        rc = pkv_launch_decode_fp8(fa, head_dim, s);
    else if (pkv_decode_fp8_tma_supported(fa))
        rc = pkv_launch_decode_fp8_tma(fa, head_dim, s);
    else
        rc = head_dim == 128 ? launch_split<128>(fa, s) : launch_split<64>(fa, s);
    if (rc != PKV_OK) return rc;
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
                                        out, workspace, workspace_bytes, cache, status, fa.d);
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
    return (pkv_paged_decode_workspace_bytes(batch, num_q_heads, max_context_len, cache) + 255) &
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
