// qk_norm_rope, qk_norm_rope_kv_store: RMS norm of every q and k head and the rotation of
// its position in one pass, and the same with the k and v rows written into the cache.
//
// What it computes.  For a head x[D] of the token at position p, with weights w[D]:
//   y = x * rsqrt(mean(x^2) + eps) * w                     (y = x where there are no weights)
//   pair i < R/2 of the first R entries, (y[i], y[i + R/2]) or (y[2i], y[2i + 1]):
//   (a, b) -> m (a cos t - b sin t, b cos t + a sin t),  t = p * w_i
// With the row's r = rsqrt(mean(x^2) + eps) outside, entry e is
//   r * (A[e] * x[e] + B[e] * x[partner of e]),
// where A and B hold the weights, the cosines and sines and m: two tables of D entries
// that depend on the token alone and serve all of its heads.
//
// Angles.  p * w_i in 32 bits is off by radians at far positions.  A frequency is held as
// the fraction of a turn it adds for each position, in units of 2^-64 turn: p times it,
// modulo 2^64, is the angle's fraction of a turn to p * 2^-65, by one integer product.  The
// nearest quarter turn is taken off as an integer, so that the rest, within 1/8 turn, goes
// to sincospi with 24 significant bits of its own.
//
// Bound: every row is read once and written once.
//
// Layout.  A CTA takes one token.  Its first threads build the tables while the rows'
// loads are in flight.  A head is D / 8 lanes of a warp (in a group of 8, 16 or 32) of 8
// entries each: 16 bytes for 16-bit types.  The half layout's partner entries come from
// the lane R/16 further on by shuffles of the packed rows, or from memory where R is no
// multiple of 16; the interleaved layout's lie in the same lane.
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;                    // heads a lane has in flight
constexpr int kMaxDim = 256;

struct HeadArgs {
    const void* in[3];                       // q, k, v
    int64_t in_stride[3];                    // elements between tokens
    void* out[2];                            // q, k (k: may be null with a cache)
    int64_t out_stride[2];
    const void* weight[2];                   // q, k; null: no norm
    int32_t weight_type;
    const int32_t* positions;
    const uint64_t* turns;
    int32_t rotary_dim, interleaved;
    float magnitude, eps;
    int32_t num_tokens, Hq, Hkv, D;
    // the cache
    const int32_t* slots;
    __nv_bfloat16* cache[2];
    int64_t num_slots;
    uint32_t* status;
};

// Where a lane finds the partner entries of its eight: nowhere (no rotation), among
// them, in another lane, in memory.
enum Partner : int { kNone, kPairs, kLane, kMemory };

template <typename T>
struct Eight;
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = pkv::ld_stream16f(p);
        b = pkv::ld_stream16f(p + 4);
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ Eight from(int lane) const {
        Eight r;
        r.a = make_float4(__shfl_sync(~0u, a.x, lane), __shfl_sync(~0u, a.y, lane),
                          __shfl_sync(~0u, a.z, lane), __shfl_sync(~0u, a.w, lane));
        r.b = make_float4(__shfl_sync(~0u, b.x, lane), __shfl_sync(~0u, b.y, lane),
                          __shfl_sync(~0u, b.z, lane), __shfl_sync(~0u, b.w, lane));
        return r;
    }
    static __device__ __forceinline__ void store(float* p, const float (&y)[8]) {
        *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(y[4], y[5], y[6], y[7]);
    }
    __device__ __forceinline__ void put(float* p) const {
        *reinterpret_cast<float4*>(p) = a;
        *reinterpret_cast<float4*>(p + 4) = b;
    }
};

__device__ __forceinline__ float2 two(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 two(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, __nv_bfloat16) {
    return pkv::pack_bf16(lo, hi);
}
__device__ __forceinline__ uint32_t pack(float lo, float hi, __half) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename T>
struct Eight {
    uint4 v;
    __device__ __forceinline__ void load(const T* p) { v = pkv::ld_stream16(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = two(w[i], T());
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    __device__ __forceinline__ Eight from(int lane) const {
        Eight r;
        r.v = make_uint4(__shfl_sync(~0u, v.x, lane), __shfl_sync(~0u, v.y, lane),
                         __shfl_sync(~0u, v.z, lane), __shfl_sync(~0u, v.w, lane));
        return r;
    }
    static __device__ __forceinline__ void store(T* p, const float (&y)[8]) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack(y[0], y[1], T()), pack(y[2], y[3], T()), pack(y[4], y[5], T()),
                       pack(y[6], y[7], T()));
    }
    __device__ __forceinline__ void put(T* p) const { *reinterpret_cast<uint4*>(p) = v; }
};

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }

__device__ __forceinline__ float weight_at(const HeadArgs& a, int which, int e) {
    const void* w = a.weight[which];
    if (w == nullptr) return 1.f;
    return a.weight_type == PKV_FP32   ? ((const float*)w)[e]
           : a.weight_type == PKV_BF16 ? __bfloat162float(((const __nv_bfloat16*)w)[e])
                                       : __half2float(((const __half*)w)[e]);
}

// cos and sin of `turns` * 2^-64 turns.
__device__ __forceinline__ void turn(uint64_t turns, float& c, float& s) {
    const uint32_t quarter = (uint32_t)((turns + (1ull << 61)) >> 62) & 3;
    const int64_t rest = (int64_t)(turns - ((uint64_t)quarter << 62));   // within 1/8 turn
    float s0, c0;
    sincospif((float)rest * 0x1p-63f, &s0, &c0);
    const float a = quarter & 1 ? s0 : c0, b = quarter & 1 ? c0 : s0;
    c = quarter == 1 || quarter == 2 ? -a : a;
    s = quarter >= 2 ? -b : b;
}

// The tables A and B of a token, for q ([0]) and for k ([1]).
struct Tables {
    float a[2][kMaxDim], b[2][kMaxDim];
};

__device__ __forceinline__ void fill_tables(const HeadArgs& g, int32_t token, Tables& t) {
    const int half = g.rotary_dim / 2;
    for (int i = threadIdx.x; i < half; i += kThreads) {
        const uint64_t p = (uint64_t)(int64_t)__ldg(g.positions + token);
        float c, s;
        turn(p * __ldg((const unsigned long long*)g.turns + i), c, s);
        c *= g.magnitude;
        s *= g.magnitude;
        const int e1 = g.interleaved ? 2 * i : i, e2 = g.interleaved ? 2 * i + 1 : i + half;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const float w1 = weight_at(g, which, e1), w2 = weight_at(g, which, e2);
            t.a[which][e1] = w1 * c;
            t.b[which][e1] = -w2 * s;
            t.a[which][e2] = w2 * c;
            t.b[which][e2] = w1 * s;
        }
    }
    for (int e = g.rotary_dim + threadIdx.x; e < g.D; e += kThreads)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            t.a[which][e] = weight_at(g, which, e);
            t.b[which][e] = 0.f;
        }
}

// kLanes: lanes of a head (8 kLanes >= D).  kStore: k and v rows go into the cache.
template <typename T, int kLanes, Partner kPartner, bool kStore>
__global__ void __launch_bounds__(kThreads) head_kernel(const HeadArgs g) {
    constexpr int kHeads = kThreads / kLanes;            // heads of a pass
    __shared__ __align__(16) Tables tab;
    const int32_t token = blockIdx.x;
    const int c = threadIdx.x % kLanes, lane = threadIdx.x & 31;
    const bool in_row = c * 8 < g.D;
    const int32_t qk = g.Hq + g.Hkv, heads = kStore ? qk + g.Hkv : qk;
    const int half = g.rotary_dim / 2;
    // the half layout's partner lane (in whole chunks)
    const int away = half / 8;
    const int other = lane + (c < away ? away : c < 2 * away ? -away : 0);
    int32_t slot = -1;
    if constexpr (kStore) {
        slot = __ldg(g.slots + token);
        if ((int64_t)slot >= g.num_slots) {
            if (threadIdx.x == 0) pkv::report(g.status, PKV_STATUS_SLOT_OUT_OF_RANGE);
            slot = -1;
        }
    }
    for (int32_t base = 0; base < heads; base += kBatch * kHeads) {
        Eight<T> x[kBatch];
        float xp[kPartner == kMemory ? kBatch : 1][8];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int32_t h = base + u * kHeads + threadIdx.x / kLanes;
            x[u] = Eight<T>{};
            if (h < heads && in_row) {
                const int which = h < g.Hq ? 0 : h < qk ? 1 : 2;
                const int32_t hh = h - (which == 0 ? 0 : which == 1 ? g.Hq : qk);
                const T* row = (const T*)g.in[which] + token * g.in_stride[which] +
                               (int64_t)hh * g.D;
                x[u].load(row + c * 8);
                if constexpr (kPartner == kMemory)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int e = c * 8 + k;
                        xp[u][k] = e < half             ? as_float(row[e + half])
                                   : e < g.rotary_dim ? as_float(row[e - half])
                                                      : 0.f;
                    }
            }
        }
        if (base == 0) {
            fill_tables(g, token, tab);
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (base + u * kHeads >= heads) break;           // alike in every thread
            const int32_t h = base + u * kHeads + threadIdx.x / kLanes;
            const int which = h < g.Hq ? 0 : 1;
            float y[8], p[8], o[8];
            x[u].get(y);
            float ss = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) ss = fmaf(y[k], y[k], ss);
#pragma unroll
            for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(~0u, ss, off);
            const float r = g.weight[which] ? rsqrtf(ss / (float)g.D + g.eps) : 1.f;
            if constexpr (kPartner == kLane) x[u].from(other).get(p);
            __syncwarp();                    // the row is read: it may be written in place
            if (h >= heads || !in_row) continue;
            if (kStore && h >= qk) {         // a v row, as it is
                if (slot >= 0)
                    x[u].put((T*)g.cache[1] + ((int64_t)slot * g.Hkv + (h - qk)) * g.D + c * 8);
                continue;
            }
            const float* ta = tab.a[which] + c * 8;
            const float* tb = tab.b[which] + c * 8;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                o[k] = ta[k] * y[k];
                if constexpr (kPartner != kNone) {
                    const float partner = kPartner == kPairs  ? y[k ^ 1]
                                          : kPartner == kLane ? p[k]
                                                              : xp[kPartner == kMemory ? u : 0][k];
                    // entries behind the rotated ones have none
                    if (c * 8 + k < g.rotary_dim) o[k] = fmaf(tb[k], partner, o[k]);
                }
                o[k] *= r;
            }
            const int32_t hh = which ? h - g.Hq : h;
            if (g.out[which])
                Eight<T>::store((T*)g.out[which] + token * g.out_stride[which] +
                                    (int64_t)hh * g.D + c * 8,
                                o);
            if (kStore && which == 1 && slot >= 0)
                Eight<T>::store((T*)g.cache[0] + ((int64_t)slot * g.Hkv + hh) * g.D + c * 8, o);
        }
    }
}

template <typename T, int kLanes, bool kStore>
int launch(const HeadArgs& g, cudaStream_t s) {
    void (*kernel)(const HeadArgs) =
        g.rotary_dim == 0        ? head_kernel<T, kLanes, kNone, kStore>
        : g.interleaved          ? head_kernel<T, kLanes, kPairs, kStore>
        : g.rotary_dim % 16 == 0 ? head_kernel<T, kLanes, kLane, kStore>
                                 : head_kernel<T, kLanes, kMemory, kStore>;
    kernel<<<(unsigned)g.num_tokens, kThreads, 0, s>>>(g);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <typename T, bool kStore>
int launch(const HeadArgs& g, cudaStream_t s) {
    return g.D <= 64    ? launch<T, 8, kStore>(g, s)
           : g.D <= 128 ? launch<T, 16, kStore>(g, s)
                        : launch<T, 32, kStore>(g, s);
}

// A [tokens, heads, D] view whose tokens are `stride` elements apart.
struct View {
    const void* p;
    int64_t stride, row;                     // row: elements of a token
};

bool overlap(const View& x, const View& y, int64_t tokens, int size) {
    const int64_t px = (int64_t)(uintptr_t)x.p, py = (int64_t)(uintptr_t)y.p;
    const int64_t ex = px + ((tokens - 1) * x.stride + x.row) * size;
    const int64_t ey = py + ((tokens - 1) * y.stride + y.row) * size;
    if (ex <= py || ey <= px) return false;
    if (x.stride != y.stride || tokens == 1) return true;
    // columns of the same packed rows
    const int64_t pitch = x.stride * size;
    const int64_t at = (((py - px) % pitch) + pitch) % pitch;
    return at < x.row * size || at + y.row * size > pitch;
}

// The checks both calls share; fills g's rows, weights, positions and rotation.
int make_args(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int32_t type,
              const void* q_weight, const void* k_weight, int32_t weight_type, float eps,
              const int32_t* positions, const pkv_rotary& rotary, int32_t num_tokens,
              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, void* q_out,
              int64_t q_out_stride, void* k_out, int64_t k_out_stride, bool need_k_out,
              HeadArgs& g) {
    if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0) return PKV_ERR_BAD_DIMENSION;
    if ((int64_t)num_q_heads + 2 * (int64_t)num_kv_heads > INT32_MAX / kMaxDim)
        return PKV_ERR_BAD_DIMENSION;
    if (head_dim <= 0 || head_dim > kMaxDim || head_dim % 8 != 0)
        return PKV_ERR_UNSUPPORTED_HEAD_DIM;
    if (type < PKV_FP32 || type > PKV_FP16 || weight_type < PKV_FP32 || weight_type > PKV_FP16)
        return PKV_ERR_BAD_DIMENSION;
    if (rotary.rotary_dim < 0 || rotary.rotary_dim > head_dim || rotary.rotary_dim % 2 != 0)
        return PKV_ERR_BAD_DIMENSION;
    if (rotary.rotary_dim > 0 && !isfinite(rotary.magnitude)) return PKV_ERR_BAD_DIMENSION;
    if ((q_weight || k_weight) && !(eps >= 0.f && isfinite(eps))) return PKV_ERR_BAD_DIMENSION;
    if (rotary.rotary_dim == 0 && !q_weight && !k_weight) return PKV_ERR_BAD_DIMENSION;
    if (num_tokens == 0) return PKV_OK;
    if (!q || !k || !q_out || (need_k_out && !k_out)) return PKV_ERR_NULL_POINTER;
    if (rotary.rotary_dim > 0 && (!positions || !rotary.turns)) return PKV_ERR_NULL_POINTER;
    const int size = type == PKV_FP32 ? 4 : 2, wsize = weight_type == PKV_FP32 ? 4 : 2;
    const int64_t q_row = (int64_t)num_q_heads * head_dim, k_row = (int64_t)num_kv_heads * head_dim;
    if (num_tokens == 1) {
        q_stride = q_out_stride = q_row;
        k_stride = k_out_stride = k_row;
    }
    if (q_stride < q_row || k_stride < k_row || q_out_stride < q_row ||
        (k_out && k_out_stride < k_row))
        return PKV_ERR_BAD_DIMENSION;
    const uintptr_t rows = (uintptr_t)q | (uintptr_t)k | (uintptr_t)q_out | (uintptr_t)k_out;
    const int64_t strides = q_stride | k_stride | q_out_stride | (k_out ? k_out_stride : 0);
    if ((rows & 15) || (strides * size) % 16 != 0) return PKV_ERR_MISALIGNED;
    if (((uintptr_t)q_weight | (uintptr_t)k_weight) & (wsize - 1)) return PKV_ERR_MISALIGNED;
    if (rotary.rotary_dim > 0 && (((uintptr_t)positions & 3) || ((uintptr_t)rotary.turns & 7)))
        return PKV_ERR_MISALIGNED;
    // an output may be its own input; no other overlap
    const View vq{q, q_stride, q_row}, vk{k, k_stride, k_row}, oq{q_out, q_out_stride, q_row},
        ok{k_out, k_out_stride, k_row};
    if (!(q_out == q && q_out_stride == q_stride) && overlap(oq, vq, num_tokens, size))
        return PKV_ERR_UNSUPPORTED;
    if (overlap(oq, vk, num_tokens, size)) return PKV_ERR_UNSUPPORTED;
    if (k_out) {
        if (!(k_out == k && k_out_stride == k_stride) && overlap(ok, vk, num_tokens, size))
            return PKV_ERR_UNSUPPORTED;
        if (overlap(ok, vq, num_tokens, size) || overlap(ok, oq, num_tokens, size))
            return PKV_ERR_UNSUPPORTED;
    }
    g = HeadArgs{};
    g.in[0] = q;
    g.in[1] = k;
    g.in_stride[0] = q_stride;
    g.in_stride[1] = k_stride;
    g.out[0] = q_out;
    g.out[1] = k_out;
    g.out_stride[0] = q_out_stride;
    g.out_stride[1] = k_out_stride;
    g.weight[0] = q_weight;
    g.weight[1] = k_weight;
    g.weight_type = weight_type;
    g.positions = positions;
    g.turns = rotary.turns;
    g.rotary_dim = rotary.rotary_dim;
    g.interleaved = rotary.interleaved != 0;
    g.magnitude = rotary.magnitude;
    g.eps = eps;
    g.num_tokens = num_tokens;
    g.Hq = num_q_heads;
    g.Hkv = num_kv_heads;
    g.D = head_dim;
    return PKV_OK;
}

}  // namespace

extern "C" int pkv_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                int32_t type, const void* q_weight, const void* k_weight,
                                int32_t weight_type, float eps, const int32_t* positions,
                                pkv_rotary rotary, int32_t num_tokens, int32_t num_q_heads,
                                int32_t num_kv_heads, int32_t head_dim, void* q_out,
                                int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                void* stream) {
    HeadArgs g;
    const int rc = make_args(q, q_stride, k, k_stride, type, q_weight, k_weight, weight_type, eps,
                             positions, rotary, num_tokens, num_q_heads, num_kv_heads, head_dim,
                             q_out, q_out_stride, k_out, k_out_stride, true, g);
    if (rc != PKV_OK || num_tokens == 0) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    return type == PKV_FP32   ? launch<float, false>(g, s)
           : type == PKV_BF16 ? launch<__nv_bfloat16, false>(g, s)
                              : launch<__half, false>(g, s);
}

extern "C" int pkv_qk_norm_rope_kv_store(
        const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
        int64_t v_stride, const void* q_weight, const void* k_weight, int32_t weight_type,
        float eps, const int32_t* positions, pkv_rotary rotary, const int32_t* slot_mapping,
        int32_t num_tokens, int32_t num_q_heads, void* q_out, int64_t q_out_stride, void* k_out,
        int64_t k_out_stride, void* k_cache, void* v_cache, pkv_cache_desc cache,
        uint32_t* status, void* stream) {
    if (cache.num_blocks <= 0 || cache.block_size <= 0) return PKV_ERR_BAD_DIMENSION;
    HeadArgs g;
    const int rc = make_args(q, q_stride, k, k_stride, PKV_BF16, q_weight, k_weight, weight_type,
                             eps, positions, rotary, num_tokens, num_q_heads, cache.num_kv_heads,
                             cache.head_dim, q_out, q_out_stride, k_out, k_out_stride, false, g);
    if (rc != PKV_OK || num_tokens == 0) return rc;
    if (!v || !k_cache || !v_cache || !slot_mapping) return PKV_ERR_NULL_POINTER;
    const int64_t row = (int64_t)g.Hkv * g.D;
    if (num_tokens == 1) v_stride = row;
    if (v_stride < row) return PKV_ERR_BAD_DIMENSION;
    if (((uintptr_t)v | (uintptr_t)k_cache | (uintptr_t)v_cache) & 15 || v_stride % 8 != 0 ||
        ((uintptr_t)slot_mapping & 3))
        return PKV_ERR_MISALIGNED;
    const View vv{v, v_stride, row};
    if (overlap({q_out, g.out_stride[0], (int64_t)g.Hq * g.D}, vv, num_tokens, 2) ||
        (k_out && overlap({k_out, g.out_stride[1], row}, vv, num_tokens, 2)))
        return PKV_ERR_UNSUPPORTED;
    g.in[2] = v;
    g.in_stride[2] = v_stride;
    g.slots = slot_mapping;
    g.cache[0] = (__nv_bfloat16*)k_cache;
    g.cache[1] = (__nv_bfloat16*)v_cache;
    g.num_slots = (int64_t)cache.num_blocks * cache.block_size;
    g.status = status;
    return launch<__nv_bfloat16, true>(g, (cudaStream_t)stream);
}

// ---------------------------------------------------------------------------
// Frequencies (host only).
// ---------------------------------------------------------------------------
extern "C" int pkv_rotary_frequencies(int32_t rotary_dim, double base, pkv_rotary_scaling scaling,
                                      double* frequencies, float* magnitude) {
    if (!frequencies || !magnitude) return PKV_ERR_NULL_POINTER;
    const double f = scaling.factor, pi2 = 6.283185307179586476925;
    const double old = (double)scaling.original_max_position;
    if (rotary_dim <= 0 || rotary_dim > kMaxDim || rotary_dim % 2 != 0) return PKV_ERR_BAD_DIMENSION;
    if (!(base > 1.0) || !isfinite(base)) return PKV_ERR_BAD_DIMENSION;
    if (scaling.kind != PKV_ROPE_PLAIN && (!(f >= 1.0) || !isfinite(f)))
        return PKV_ERR_BAD_DIMENSION;
    const int32_t half = rotary_dim / 2;
    double lo = 0.0, hi = 0.0, mag = 1.0;
    switch (scaling.kind) {
        case PKV_ROPE_PLAIN:
        case PKV_ROPE_LINEAR:
            break;
        case PKV_ROPE_NTK:
            if (rotary_dim <= 2) return PKV_ERR_BAD_DIMENSION;
            base *= pow(f, (double)rotary_dim / (rotary_dim - 2));
            if (!isfinite(base)) return PKV_ERR_BAD_DIMENSION;
            break;
        case PKV_ROPE_YARN:
            if (!(old > 0.0) || !(scaling.low > 0.0) || !(scaling.high > scaling.low) ||
                !isfinite(scaling.high))
                return PKV_ERR_BAD_DIMENSION;
            // the pair that makes `high` turns in `old` positions, and the one that makes `low`
            lo = floor(half * log(old / (scaling.high * pi2)) / log(base));
            hi = ceil(half * log(old / (scaling.low * pi2)) / log(base));
            if (lo < 0.0) lo = 0.0;
            if (hi > rotary_dim - 1) hi = rotary_dim - 1;
            mag = 0.1 * log(f) + 1.0;
            break;
        case PKV_ROPE_BANDS:
            if (!(old > 0.0) || !(scaling.low > 0.0) || !(scaling.high > scaling.low) ||
                !isfinite(scaling.high))
                return PKV_ERR_BAD_DIMENSION;
            break;
        default:
            return PKV_ERR_BAD_DIMENSION;
    }
    for (int32_t i = 0; i < half; ++i) {
        const double w = pow(base, -2.0 * i / rotary_dim);
        double keep = 1.0;                                   // share of the frequency kept
        if (scaling.kind == PKV_ROPE_LINEAR) keep = 0.0;
        if (scaling.kind == PKV_ROPE_YARN)
            keep = 1.0 - (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
        if (scaling.kind == PKV_ROPE_BANDS)
            keep = (old * w / pi2 - scaling.low) / (scaling.high - scaling.low);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        frequencies[i] = keep == 1.0 ? w : w * keep + w / f * (1.0 - keep);
    }
    *magnitude = (float)mag;
    return PKV_OK;
}

extern "C" int pkv_rotary_turns(const double* frequencies, int32_t count, uint64_t* turns) {
    if (count < 0) return PKV_ERR_BAD_DIMENSION;
    if (count > 0 && (!frequencies || !turns)) return PKV_ERR_NULL_POINTER;
    // 1 / (2 pi) in units of 2^-192, most significant word first
    const uint64_t inv[3] = {0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull};
    for (int32_t i = 0; i < count; ++i)
        if (!(frequencies[i] >= 0.0 && frequencies[i] <= 65536.0)) return PKV_ERR_BAD_DIMENSION;
    for (int32_t i = 0; i < count; ++i) {
        int e = 0;
        const double m = frexp(frequencies[i], &e);          // frequency = m 2^e
        const uint64_t mant = (uint64_t)ldexp(m, 53);
        // mant * inv: four words, in units of 2^(e - 53 - 192)
        uint64_t w[4];                                       // least significant first
        unsigned __int128 carry = 0;
        for (int j = 0; j < 3; ++j) {
            carry += (unsigned __int128)mant * inv[2 - j];
            w[j] = (uint64_t)carry;
            carry >>= 64;
        }
        w[3] = (uint64_t)carry;
        // the fraction in units of 2^-64, rounded: shifted right by 181 - e, which is 164 at
        // least (e <= 17)
        const int shift = 181 - e;
        uint64_t out = 0;
        for (int b = 0; b < 64; ++b) {
            const int from = shift + b;
            if (from < 256 && (w[from >> 6] >> (from & 63)) & 1) out |= 1ull << b;
        }
        const int below = shift - 1;
        if (below < 256 && (w[below >> 6] >> (below & 63)) & 1) ++out;
        turns[i] = out;
    }
    return PKV_OK;
}
