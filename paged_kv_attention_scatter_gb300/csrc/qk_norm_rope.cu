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

constexpr int kThreads = 192;
constexpr int kBatch = 2;                    // heads a lane has in flight
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
    float magnitude, eps, inv_dim;           // inv_dim: 1 / D
    int32_t num_tokens, Hq, Hkv, D;
    // the cache
    const int32_t* slots;
    __nv_bfloat16* cache[2];
    int64_t num_slots;
    uint32_t* status;
};

// Where a lane finds the partner entries of its sixteen: nowhere (no rotation), next to
// them, at the same place of its other chunk, or through shared memory.
enum Partner : int { kNone, kPairs, kChunks, kShared };

// Eight entries as four packed pairs of fp32; arithmetic on pairs is one instruction.
struct Pairs {
    uint64_t v[4];
};

__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 up2(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t swapped(uint64_t v) {
    const float2 f = up2(v);
    return pk2(f.y, f.x);
}

__device__ __forceinline__ uint64_t two(uint32_t w, __nv_bfloat16) {
    return pk2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint64_t two(uint32_t w, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return pk2(f.x, f.y);
}
__device__ __forceinline__ uint32_t pack(float2 f, __nv_bfloat16) {
    return pkv::pack_bf16(f.x, f.y);
}
__device__ __forceinline__ uint32_t pack(float2 f, __half) {
    const __half2 v = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight entries as they lie in memory.
template <typename T>
struct Eight {
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const T* p) { v = pkv::ld_stream16(p); }
    __device__ __forceinline__ Pairs get() const {
        return {{two(v.x, T()), two(v.y, T()), two(v.z, T()), two(v.w, T())}};
    }
    static __device__ __forceinline__ void store(T* p, const Pairs& y) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack(up2(y.v[0]), T()), pack(up2(y.v[1]), T()), pack(up2(y.v[2]), T()),
                       pack(up2(y.v[3]), T()));
    }
    __device__ __forceinline__ void put(T* p) const { *reinterpret_cast<uint4*>(p) = v; }
};
template <>
struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float* p) {
        a = pkv::ld_stream16f(p);
        b = pkv::ld_stream16f(p + 4);
    }
    __device__ __forceinline__ Pairs get() const {
        return {{pk2(a.x, a.y), pk2(a.z, a.w), pk2(b.x, b.y), pk2(b.z, b.w)}};
    }
    static __device__ __forceinline__ void store(float* p, const Pairs& y) {
        const float2 f0 = up2(y.v[0]), f1 = up2(y.v[1]), f2 = up2(y.v[2]), f3 = up2(y.v[3]);
        *reinterpret_cast<float4*>(p) = make_float4(f0.x, f0.y, f1.x, f1.y);
        *reinterpret_cast<float4*>(p + 4) = make_float4(f2.x, f2.y, f3.x, f3.y);
    }
    __device__ __forceinline__ void put(float* p) const {
        *reinterpret_cast<float4*>(p) = a;
        *reinterpret_cast<float4*>(p + 4) = b;
    }
};

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

// Half of the threads fill q's, half k's: each its own cosines and sines, for a token's rows wait
// for the slowest of them.
__device__ __forceinline__ void fill_tables(const HeadArgs& g, int32_t token, Tables& t) {
    const int half = g.rotary_dim / 2, which = threadIdx.x >= kThreads / 2;
    const int first = threadIdx.x - which * (kThreads / 2);
    float *ta = t.a[which], *tb = t.b[which];
    if (half > 0) {
        const uint64_t p = (uint64_t)(int64_t)__ldg(g.positions + token);
        for (int i = first; i < half; i += kThreads / 2) {
            const int e1 = g.interleaved ? 2 * i : i, e2 = g.interleaved ? 2 * i + 1 : i + half;
            const float w1 = weight_at(g, which, e1), w2 = weight_at(g, which, e2);
            float c, s;
            turn(p * __ldg((const unsigned long long*)g.turns + i), c, s);
            c *= g.magnitude;
            s *= g.magnitude;
            ta[e1] = w1 * c;
            tb[e1] = -w2 * s;
            ta[e2] = w2 * c;
            tb[e2] = w1 * s;
        }
    }
    for (int e = g.rotary_dim + first; e < g.D; e += kThreads / 2) {
        ta[e] = weight_at(g, which, e);
        tb[e] = 0.f;
    }
}

__device__ __forceinline__ Pairs table_at(const float* p) {
    const ulonglong2 lo = *reinterpret_cast<const ulonglong2*>(p);
    const ulonglong2 hi = *reinterpret_cast<const ulonglong2*>(p + 4);
    return {{lo.x, lo.y, hi.x, hi.y}};
}

// r (A x + B x') of eight entries from e0 on; `rotated` of them have a partner.
template <Partner kPartner>
__device__ __forceinline__ Pairs turned(const float* a, const float* b, const Pairs& x,
                                        const Pairs& partner, int e0, int rotary_dim,
                                        uint64_t r2) {
    const Pairs ta = table_at(a + e0);
    Pairs y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y.v[i] = mul2(ta.v[i], x.v[i]);
    if constexpr (kPartner != kNone) {
        // entries behind the rotated ones have none: an infinite one beside them, times
        // the table's zero, would make them NaN
        if (e0 < rotary_dim) {
            const Pairs tb = table_at(b + e0);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (e0 + 2 * i < rotary_dim) y.v[i] = fma2(tb.v[i], partner.v[i], y.v[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y.v[i] = mul2(y.v[i], r2);
    return y;
}

// kLanes: lanes of a head (16 kLanes >= D), each with two chunks of eight entries.
// kStore: k and v rows go into the cache.
template <typename T, int kLanes, Partner kPartner, bool kStore>
__global__ void __launch_bounds__(kThreads) head_kernel(const HeadArgs g) {
    constexpr int kHeads = kThreads / kLanes;            // heads of a pass
    __shared__ __align__(16) Tables tab;
    // a pass's rows as fp32, for partners that lie across chunks
    __shared__ __align__(16) float rows[kPartner == kShared ? kThreads * 16 : 1];
    const int32_t token = blockIdx.x;
    const int j = threadIdx.x % kLanes, head = threadIdx.x / kLanes;
    const int32_t qk = g.Hq + g.Hkv, heads = kStore ? qk + g.Hkv : qk;
    // this lane's chunks: where they are partners (half layout, whole chunks) chunk j and
    // the one half the rotated part away, and behind those as elsewhere: j and j + as many
    // as there are lanes with a first chunk
    const int chunks = g.D / 8, away = kPartner == kChunks ? g.rotary_dim / 16 : 0;
    const int left = chunks - 2 * away;                  // chunks not in such pairs
    const int c0 = j < away ? j : j + away, c1 = j < away ? j + away : j + away + (left + 1) / 2;
    const bool has0 = j < away + (left + 1) / 2;
    const bool has1 = j < away || (has0 && c1 < chunks);
    const int e0 = c0 * 8, e1 = has1 ? c1 * 8 : 0;
    int32_t slot = -1;
    if constexpr (kStore) {
        slot = __ldg(g.slots + token);
        if ((int64_t)slot >= g.num_slots) {
            if (threadIdx.x == 0) pkv::report(g.status, PKV_STATUS_SLOT_OUT_OF_RANGE);
            slot = -1;
        }
    }
    for (int32_t base = 0; base < heads; base += kBatch * kHeads) {
        Eight<T> x0[kBatch], x1[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int32_t h = base + u * kHeads + head;
            x0[u].zero();
            x1[u].zero();
            if (h < heads) {
                const int which = h < g.Hq ? 0 : h < qk ? 1 : 2;
                const int32_t hh = h - (which == 0 ? 0 : which == 1 ? g.Hq : qk);
                const T* row = (const T*)g.in[which] + token * g.in_stride[which] +
                               (int64_t)hh * g.D;
                if (has0) x0[u].load(row + e0);
                if (has1) x1[u].load(row + e1);
            }
        }
        if (base == 0) {
            fill_tables(g, token, tab);
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (base + u * kHeads >= heads) break;           // alike in every thread
            const int32_t h = base + u * kHeads + head;
            if (kStore && h >= qk) {                         // a v row, as it is
                if (slot >= 0 && h < heads) {
                    T* to = (T*)g.cache[1] + ((int64_t)slot * g.Hkv + (h - qk)) * g.D;
                    if (has0) x0[u].put(to + e0);
                    if (has1) x1[u].put(to + e1);
                }
            }
            if (kStore && __all_sync(~0u, h >= qk)) continue;
            const int which = h < g.Hq ? 0 : 1;
            const Pairs a = x0[u].get(), b = x1[u].get();
            float r = 1.f;
            if (g.weight[0] || g.weight[1]) {
                uint64_t s2 = mul2(a.v[0], a.v[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i) s2 = fma2(a.v[i], a.v[i], s2);
#pragma unroll
                for (int i = 0; i < 4; ++i) s2 = fma2(b.v[i], b.v[i], s2);
                const float2 s = up2(s2);
                float ss = s.x + s.y;
#pragma unroll
                for (int off = kLanes / 2; off > 0; off >>= 1)
                    ss += __shfl_xor_sync(~0u, ss, off);
                if (g.weight[which]) r = rsqrtf(ss * g.inv_dim + g.eps);
            }
            const uint64_t r2 = pk2(r, r);
            Pairs pa = a, pb = b;                            // partners
            if constexpr (kPartner == kPairs) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    pa.v[i] = swapped(a.v[i]);
                    pb.v[i] = swapped(b.v[i]);
                }
            } else if constexpr (kPartner == kChunks) {
                pa = b;
                pb = a;
            } else if constexpr (kPartner == kShared) {
                float* mine = rows + head * (kLanes * 16);
                const int half = g.rotary_dim / 2;
                __syncwarp();                                // the last rows are read
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (has0) *reinterpret_cast<uint64_t*>(mine + e0 + 2 * i) = a.v[i];
                    if (has1) *reinterpret_cast<uint64_t*>(mine + e1 + 2 * i) = b.v[i];
                }
                __syncwarp();
                if (half % 4 == 0) {         // four entries have their partners in a row
                    auto at = [&](int e, Pairs& to, int i) {
                        ulonglong2 v = make_ulonglong2(0, 0);
                        if (e < g.rotary_dim)
                            v = *reinterpret_cast<const ulonglong2*>(
                                mine + (e < half ? e + half : e - half));
                        to.v[i] = v.x;
                        to.v[i + 1] = v.y;
                    };
                    at(e0, pa, 0);
                    at(e0 + 4, pa, 2);
                    at(e1, pb, 0);
                    at(e1 + 4, pb, 2);
                } else {
                    auto at = [&](int e) {
                        return e < half ? mine[e + half] : e < g.rotary_dim ? mine[e - half] : 0.f;
                    };
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        pa.v[i] = pk2(at(e0 + 2 * i), at(e0 + 2 * i + 1));
                        pb.v[i] = pk2(at(e1 + 2 * i), at(e1 + 2 * i + 1));
                    }
                }
            }
            __syncwarp();                    // the rows are read: they may be written in place
            if (h >= qk || !has0) continue;
            const int32_t hh = which ? h - g.Hq : h;
            const Pairs y0 = turned<kPartner>(tab.a[which], tab.b[which], a, pa, e0,
                                              g.rotary_dim, r2);
            const Pairs y1 = turned<kPartner>(tab.a[which], tab.b[which], b, pb, e1,
                                              g.rotary_dim, r2);
            if (g.out[which]) {
                T* to = (T*)g.out[which] + token * g.out_stride[which] + (int64_t)hh * g.D;
                Eight<T>::store(to + e0, y0);
                if (has1) Eight<T>::store(to + e1, y1);
            }
            if (kStore && which == 1 && slot >= 0) {
                T* to = (T*)g.cache[0] + ((int64_t)slot * g.Hkv + hh) * g.D;
                Eight<T>::store(to + e0, y0);
                if (has1) Eight<T>::store(to + e1, y1);
            }
        }
    }
}

template <typename T, int kLanes, bool kStore>
int launch(const HeadArgs& g, cudaStream_t s) {
    void (*kernel)(const HeadArgs) =
        g.rotary_dim == 0        ? head_kernel<T, kLanes, kNone, kStore>
        : g.interleaved          ? head_kernel<T, kLanes, kPairs, kStore>
        : g.rotary_dim % 16 == 0 ? head_kernel<T, kLanes, kChunks, kStore>
                                 : head_kernel<T, kLanes, kShared, kStore>;
    kernel<<<(unsigned)g.num_tokens, kThreads, 0, s>>>(g);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <typename T, bool kStore>
int launch(const HeadArgs& g, cudaStream_t s) {
    return g.D <= 64    ? launch<T, 4, kStore>(g, s)
           : g.D <= 128 ? launch<T, 8, kStore>(g, s)
                        : launch<T, 16, kStore>(g, s);
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
    g.inv_dim = 1.f / (float)head_dim;
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
