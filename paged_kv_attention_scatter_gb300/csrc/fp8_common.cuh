// Shared pieces of the 8-bit KV cache: e4m3 codes with one fp32 scale for each
// (cache block, kv head), value = code * scale.
#pragma once

#include "decode_common.cuh"

namespace pkv {

constexpr float kFp8Max = 448.f;             // largest e4m3 value, 1.75 * 2^8
constexpr int kFp8MaxBlockSize = 1024;       // largest cache block (see kv_store_fp8.cu)
// Scales the library writes are powers of two with an exponent in this range:
// 448 * 2^119 is still finite in fp32, and anything below 448 * 2^-64 is zero
// for attention.
constexpr int kScaleExpLo = -64, kScaleExpHi = 119;

// A scale that attention can use.  The lower bound keeps 1 / scale, summed
// over any number of keys, finite in fp32.
__device__ __forceinline__ bool scale_ok(float s) {
    return s >= 7.888609052210118e-31f && s <= 3.4028234663852886e38f;   // [2^-100, max]
}

// Two e4m3 codes (low byte first) -> f16x2.  Exact: every e4m3 value is an f16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
    return r;
}

// Both halves of a word of four codes.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    uint16_t a, b;
    asm("mov.b32 {%0, %1}, %2;" : "=h"(a), "=h"(b) : "r"(codes));
    lo = e4m3x2_to_f16x2(a);
    hi = e4m3x2_to_f16x2(b);
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
    float2 f;
    asm("{ .reg .b16 a, b;\n"
        "  mov.b32 {a, b}, %2;\n"
        "  cvt.f32.f16 %0, a;\n"
        "  cvt.f32.f16 %1, b; }"
        : "=f"(f.x), "=f"(f.y)
        : "r"(h));
    return f;
}

// Two floats -> two e4m3 codes, `lo` in the low byte: nearest, ties to even,
// magnitudes above 448 (infinities too) become 448, NaN stays NaN.
__device__ __forceinline__ uint16_t float2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// D = A*B + D for one m16n8k16 f16 tile with fp32 accumulation.
__device__ __forceinline__ void mma_f16_16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two floats -> packed f16x2 (round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One lane's share of a q row as f16 A fragments for S = Q K^T against codes:
// k-step kk = 4i + w holds head_dim entries 16 * (t + 4i) + 4w .. + 3, the codes
// of word w of a lane's i-th 16-byte chunk of a K row.  The row is multiplied by
// a power of two that brings its largest finite entry to [2^14, 2^15) (f16 has
// less range than bf16) and the inverse power is returned.  The four lanes of a
// row call it together; `live` false gives zeros.
template <int D>
__device__ __forceinline__ float load_q_f16(const __nv_bfloat16* row, bool live, int t,
                                            uint32_t qa[D / 16][2]) {
    uint32_t raw[D / 16][2];
    uint32_t mag = 0;
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (live) w = *reinterpret_cast<const uint4*>(row + 16 * (t + 4 * i) + 8 * half);
            raw[4 * i + 2 * half][0] = w.x;
            raw[4 * i + 2 * half][1] = w.y;
            raw[4 * i + 2 * half + 1][0] = w.z;
            raw[4 * i + 2 * half + 1][1] = w.w;
        }
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t lo = raw[kk][e] & 0x7fffu, hi = (raw[kk][e] >> 16) & 0x7fffu;
            mag = max(mag, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
    // largest entry 1.f * 2^(E - 127): multiply by 2^(14 - (E - 127)), kept where
    // it and its inverse are normal fp32 numbers
    const int e = min(max(14 - ((int)(mag >> 7) - 127), -113), 113);
    const float up = __int_as_float((e + 127) << 23);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            qa[kk][j] = pack_f16(__int_as_float((int)(raw[kk][j] << 16)) * up,
                                 __int_as_float((int)(raw[kk][j] & 0xffff0000u)) * up);
    return __int_as_float((127 - e) << 23);
}

// One paged_decode over an e4m3 cache.  `d` holds the batch, the chunk
// schedule and the outputs as in the bf16 decode (its cache pointers unused).
struct Fp8DecodeArgs {
    DecodeArgs d;
    const uint8_t* kc;
    const uint8_t* vc;
    const float* ks;                 // [num_blocks, num_kv_heads]
    const float* vs;
};

}  // namespace pkv

// The TMA split kernel (paged_decode_fp8_tma.cu): whether the shapes are its own,
// and its launch as a programmatic dependent of the plan kernel.
bool pkv_decode_fp8_tma_supported(const pkv::Fp8DecodeArgs& fa);
int pkv_launch_decode_fp8_tma(const pkv::Fp8DecodeArgs& fa, int head_dim, cudaStream_t s);

// The tcgen05 split kernel (paged_decode_fp8_tc.cu) for head_dim 128, likewise.
int pkv_launch_decode_fp8(const pkv::Fp8DecodeArgs& fa, int head_dim, cudaStream_t s);

// kv_store_fp8.cu: argument checks (enqueue nothing) and the launch.
struct Fp8StoreCall {
    const void* k;
    const void* v;
    void* k_cache;
    void* v_cache;
    float* k_scale;
    float* v_scale;
    const int32_t* slot_mapping;
    int32_t num_tokens;
    void* workspace;
    size_t workspace_bytes;
    pkv_cache_desc cache;
    uint32_t* status;
};
int pkv_kv_store_fp8_check(const Fp8StoreCall& c);
int pkv_kv_store_fp8_launch(const Fp8StoreCall& c, cudaStream_t s);
