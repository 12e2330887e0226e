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

// A scale that attention can use.  The lower bound keeps 2^8 / scale, summed
// over 2^23 keys, finite in fp32.
__device__ __forceinline__ bool scale_ok(float s) {
    return s >= 0x1p-96f && s <= 3.4028234663852886e38f;
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

// Two floats -> packed f16x2 (round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One paged_decode over an e4m3 cache.  `d` holds the batch, the chunk
// schedule and the outputs as in the bf16 decode (its cache pointers unused).
struct Fp8DecodeArgs {
    DecodeArgs d;
    const uint8_t* kc;
    const uint8_t* vc;
    const float* ks;                 // [num_blocks, num_kv_heads]
    const float* vs;
    int32_t no_combine;              // every sequence is one chunk at most: the split kernel
                                     // writes all output rows
};

}  // namespace pkv

// The split kernel (paged_decode_fp8_tc.cu), a programmatic dependent of the plan
// kernel.
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
