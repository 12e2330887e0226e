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
// Bound: every row is read once and written once; beside that, the instructions of a head.
//
// Layout.  A head is 4, 8 or 16 lanes of a warp, with two chunks of eight entries each: for
// the half layout the two that are each other's partners where the rotated part is whole
// chunks, so that no entry crosses lanes; the interleaved layout's partners lie in the same
// chunk, and the others come through shared memory, four in one access where they lie so.
// Arithmetic is on packed pairs of fp32.
//
// head_kernel, for few tokens: a CTA takes one token, all of its heads at once, and builds
// the tables while the rows' loads are in flight.  One token of 24 heads takes 2.5 us, an
// empty kernel about as long.  192 threads with two heads each in flight (in 32 bits one: 2047
// tokens of 24 heads of 80 11.5 us for 12.7), six CTAs an SM (some 16-bit forms spill 8 to 20 bytes
// there; with seven all spill and take up to 30% longer); 128 threads took 8% longer for
// 8191 such tokens, the tables built by half of the threads 15%.
//
// row_kernel, for many: an SM's 16 warps each work through a run of pieces (some heads of a
// token), with A and B in registers, made once for a token's q and once for its k, and rows
// that arrive through shared memory two pieces of 4 KB ahead.  head_kernel reads A and B from
// shared memory for every head and waits for its token's angles before any row: it is bound
// by those reads and by the wait.  row_kernel fills no pipe: it issues in 43 to 57% of the cycles
// and DRAM is busy for 32 to 63% (the rotation of 8191 tokens in 32 bits, 16384 tokens into
// the cache, 5.6 TB/s): two pieces in flight for each of 16 warps do not hide their latency.
// head / row kernel, us:
//   tokens                                         1024        2048        4096        16384
//   24 heads of 80, 32 bits, partial rotation    7.1/6.7    11.5/9.4   20.6/15.0   75.6/51.3
//   24 of 128, 32 bits, all rotated              7.4/7.5   11.3/10.1   18.0/17.6   66.6/71.8
//   40 of 128, 16 bits, pairs, half rotated      6.4/7.4     9.5/9.8   16.8/15.5   62.1/61.0
//   24 of 128, bf16, all rotated                 5.5/5.7     7.9/7.5   13.2/11.9   48.4/40.4
//   9 of 128, 16 bits, pairs, half rotated       4.3/4.4     6.1/5.6     9.9/8.2   35.0/22.3
//   48 of 128, bf16, into the cache              8.3/9.3   12.7/12.8   23.0/20.6  101.8/71.4
// One threshold for all, kManyTokens: they cross between 1000 and 2500 tokens, whatever the heads.
// (Whole rotations in 32 bits cross back: 8% at 16384 tokens are given away there.)
// Five stages of 2 KB take 1.6% less for the last and 2 to 8% more for the others at 2048 and 4096
// tokens; 20 warps with smaller stages 3% more for the last; 24 and 32 warps spill.
// Both kernels compute an entry by the same steps: a token's bits are the same in any batch.
//
// Equal slots.  Two tokens' rows in one slot could mix, 16 bytes of one and 16 of the other, so
// that the last token of a slot is found first and alone stores.  head_kernel compares its
// token's slot with those behind it; row_kernel puts its CTA's slots into a table in shared
// memory, past which all slots go once, while the first rows arrive: 0.4 us of 512 tokens,
// 2.7 of 16384.  The slots that the table has room for set the tokens of a launch, 150784 on
// 152 SMs.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "common.cuh"

namespace {

constexpr int kThreads = 192;
template <typename T>
constexpr int kBatchOf = sizeof(T) == 4 ? 1 : 2;   // heads a lane of head_kernel has in flight
constexpr int kMaxDim = 256;
constexpr int kManyTokens = 2048;            // from here on, row_kernel

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
    float tiny_unit;                         // see kLeastSquares
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

// 16 bytes past the nearest cache, by an ordinary load: the rows may be written in place.
__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// Eight entries as they lie in memory.
template <typename T>
struct Eight {
    uint4 v;
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const T* p) { v = load16(p); }
    __device__ __forceinline__ Pairs get() const {
        return {{two(v.x, T()), two(v.y, T()), two(v.z, T()), two(v.w, T())}};
    }
    __device__ __forceinline__ void take(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
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
        const uint4 u = load16(p), v = load16(p + 4);
        a = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                        __uint_as_float(u.w));
        b = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                        __uint_as_float(v.w));
    }
    __device__ __forceinline__ Pairs get() const {
        return {{pk2(a.x, a.y), pk2(a.z, a.w), pk2(b.x, b.y), pk2(b.z, b.w)}};
    }
    __device__ __forceinline__ void take(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
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

// Sums of squares that 32 bits hold with all their places.  A head whose sum lies outside (entries
// beyond 2^59, or all below 2^-50) is multiplied by a power of two first, eps by its
// square: 2^-70 brings the largest entries to 2^58, tiny_unit the small ones to 2^-49 and more
// where eps leaves room for it.  Halves cannot be so large or small.
constexpr float kLeastSquares = 0x1p-100f, kMostSquares = 0x1p126f, kHugeUnit = 0x1p-70f;
template <typename T>
constexpr bool kAnySquares = !std::is_same<T, __half>::value;

__device__ __forceinline__ bool odd_squares(float ss) {
    return !(ss >= kLeastSquares && ss < kMostSquares);
}
__device__ __forceinline__ float odd_unit(const HeadArgs& g, float ss) {
    return ss < kLeastSquares ? g.tiny_unit : kHugeUnit;
}
__device__ __forceinline__ void scale(Pairs& x, float f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x.v[i] = mul2(x.v[i], pk2(f, f));
}

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
__global__ void __launch_bounds__(kThreads, 6) head_kernel(const HeadArgs g) {
    constexpr int kHeads = kThreads / kLanes;            // heads of a pass
    constexpr int kBatch = kBatchOf<T>;
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
            // of equal slots the last token's rows are stored
            bool later = false;
            if (kStore && slot >= 0)
#pragma unroll 4
                for (int32_t t = token + 1 + threadIdx.x; t < g.num_tokens; t += kThreads)
                    later |= __ldg(g.slots + t) == slot;
            fill_tables(g, token, tab);
            if (__syncthreads_or(later)) slot = -1;
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
            Pairs a = x0[u].get(), b = x1[u].get();
            float r = 1.f;
            if (g.weight[0] || g.weight[1]) {
                float ss, eps = g.eps;
#pragma unroll 1
                for (bool scaled = false;; scaled = true) {
                    uint64_t s2 = mul2(a.v[0], a.v[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) s2 = fma2(a.v[i], a.v[i], s2);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s2 = fma2(b.v[i], b.v[i], s2);
                    const float2 s = up2(s2);
                    ss = s.x + s.y;
#pragma unroll
                    for (int off = kLanes / 2; off > 0; off >>= 1)
                        ss += __shfl_xor_sync(~0u, ss, off);
                    if (!kAnySquares<T> || scaled) break;
                    const bool odd = h < qk && g.weight[which] && odd_squares(ss);
                    if (!__any_sync(~0u, odd)) break;
                    const float f = odd ? odd_unit(g, ss) : 1.f;
                    scale(a, f);
                    scale(b, f);
                    eps = eps * f * f;
                }
                if (g.weight[which]) r = rsqrtf(fmaf(ss, g.inv_dim, eps));
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

// ---------------------------------------------------------------------------
// Many tokens: a warp works through a run of pieces, a piece being some heads of one
// token's q, k or v.
// ---------------------------------------------------------------------------
// A piece holds a pass's heads at least: 2 heads of 256 in 32 bits are 2 KB.
constexpr int kWarps = 16, kStages = 3, kPieceBytes = 4096;

struct Stage {
    uint4 rows[kPieceBytes / 16];
    int32_t position, slot, unused[2];
};

// One warp's shared memory.
struct WarpShared {
    Stage stage[kStages];
    float c[kMaxDim / 2], s[kMaxDim / 2];    // of the token's pairs
};

// The slots of a CTA's tokens and the last token of the call that has each: open addressing.
constexpr int kSlotTable = 2048, kTokensPerCta = kSlotTable / 2 - 32;

struct RowShared {
    float weight[2][kMaxDim];
    WarpShared warp[kWarps];
    int32_t slot[kSlotTable], token[kSlotTable];
};

__device__ __forceinline__ int slot_hash(int32_t slot) {
    static_assert(kSlotTable == 1 << 11, "the product's upper 11 bits");
    return (int)((uint32_t)slot * 2654435769u >> 21);
}

// Where a slot is in the table, or its first free place.
__device__ __forceinline__ int slot_place(const int32_t* table, int32_t slot) {
    int at = slot_hash(slot);
    while (table[at] != slot && table[at] >= 0) at = (at + 1) % kSlotTable;
    return at;
}

struct Pieces {
    int32_t heads, of_q, of_k, per_token;    // heads of a piece; pieces of q, of k, of a token
};

__device__ __forceinline__ void async16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void async4(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}

// Which rows a piece of a token holds: q, k or v (0, 1, 2), its first head, its heads.
struct Piece {
    int32_t which, h0, n;
};
__device__ __forceinline__ Piece piece_at(const HeadArgs& g, const Pieces& p, int32_t i) {
    const int32_t which = i < p.of_q ? 0 : i < p.of_q + p.of_k ? 1 : 2;
    const int32_t h0 = (i - (which == 0 ? 0 : which == 1 ? p.of_q : p.of_q + p.of_k)) * p.heads;
    const int32_t left = (which == 0 ? g.Hq : g.Hkv) - h0;
    return {which, h0, left < p.heads ? left : p.heads};
}

// Four entries' partners in a row, as two packed pairs.
__device__ __forceinline__ void four(const float* p, uint64_t& lo, uint64_t& hi) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    lo = v.x;
    hi = v.y;
}
template <typename T>
__device__ __forceinline__ void four(const T* p, uint64_t& lo, uint64_t& hi) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    lo = two(v.x, T());
    hi = two(v.y, T());
}

template <typename T, int kLanes, Partner kPartner, bool kStore>
__global__ void __launch_bounds__(kWarps * 32, 1) row_kernel(const HeadArgs g, const Pieces p) {
    constexpr int kHeads = 32 / kLanes, kAhead = kStages - 1;
    extern __shared__ __align__(16) unsigned char raw[];
    RowShared& sh = *reinterpret_cast<RowShared*>(raw);
    for (int i = threadIdx.x; i < 2 * g.D; i += kWarps * 32) {
        const int which = i >= g.D, e = i - which * g.D;
        sh.weight[which][e] = weight_at(g, which, e);
    }
    if (kStore)
        for (int i = threadIdx.x; i < kSlotTable; i += kWarps * 32) sh.slot[i] = sh.token[i] = -1;
    __syncthreads();
    const int lane = threadIdx.x % 32, j = lane % kLanes, head = lane / kLanes;
    WarpShared& my = sh.warp[threadIdx.x / 32];
    // this lane's chunks, as in head_kernel
    const int chunks = g.D / 8, away = kPartner == kChunks ? g.rotary_dim / 16 : 0;
    const int left = chunks - 2 * away;
    const int c0 = j < away ? j : j + away, c1 = j < away ? j + away : j + away + (left + 1) / 2;
    const bool has0 = j < away + (left + 1) / 2;
    const bool has1 = j < away || (has0 && c1 < chunks);
    const int e0 = has0 ? c0 * 8 : 0, e1 = has1 ? c1 * 8 : 0;
    const int half = g.rotary_dim / 2;

    // this warp's run of pieces
    const int64_t warps = (int64_t)gridDim.x * kWarps, w0 = (int64_t)blockIdx.x * kWarps;
    const int64_t w = w0 + threadIdx.x / 32, units = (int64_t)g.num_tokens * p.per_token;
    const int64_t first = units * w / warps;
    const int32_t count = (int32_t)(units * (w + 1) / warps - first);
    struct Cursor {
        int32_t token, at;
    };
    auto advance = [&](Cursor& c) {
        if (++c.at == p.per_token) {
            c.at = 0;
            ++c.token;
        }
    };
    Cursor now{(int32_t)(first / p.per_token), (int32_t)(first % p.per_token)};
    Cursor next = now;                       // the piece at hand, the next to ask for

    auto ask = [&](int32_t i) {
        if (i < count) {
            Stage& st = my.stage[i % kStages];
            const Piece pc = piece_at(g, p, next.at);
            const T* from = (const T*)g.in[pc.which] + next.token * g.in_stride[pc.which] +
                            (int64_t)pc.h0 * g.D;
            const int32_t vecs = pc.n * g.D * (int32_t)sizeof(T) / 16 - lane;
            const uint4* mine = (const uint4*)from + lane;
#pragma unroll
            for (int v = 0; v < kPieceBytes / 16; v += 32)
                if (v < vecs) async16(st.rows + lane + v, mine + v);
            if (lane == 0) {
                if (kPartner != kNone) async4(&st.position, g.positions + next.token);
                if (kStore) async4(&st.slot, g.slots + next.token);
            }
            advance(next);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ask(i);

    if constexpr (kStore) {
        // of equal slots the last token's rows are stored: the CTA's slots into the table, then
        // all tokens past it
        const int32_t t0 = (int32_t)(units * w0 / warps / p.per_token);
        const int32_t t1 = (int32_t)((units * (w0 + kWarps) / warps + p.per_token - 1) /
                                     p.per_token);
        for (int32_t t = t0 + threadIdx.x; t < t1; t += kWarps * 32) {
            const int32_t slot = __ldg(g.slots + t);
            if (slot < 0) continue;
            for (int at = slot_hash(slot);; at = (at + 1) % kSlotTable) {
                const int32_t had = atomicCAS(&sh.slot[at], -1, slot);
                if (had == -1 || had == slot) break;
            }
        }
        __syncthreads();
        constexpr int kBatchSlots = 8;
        for (int32_t t = t0 + threadIdx.x; t < g.num_tokens; t += kBatchSlots * kWarps * 32) {
            int32_t slot[kBatchSlots], at[kBatchSlots], key[kBatchSlots];
#pragma unroll
            for (int i = 0; i < kBatchSlots; ++i) {
                const int32_t u = t + i * kWarps * 32;
                slot[i] = u < g.num_tokens ? __ldg(g.slots + u) : -1;
            }
#pragma unroll
            for (int i = 0; i < kBatchSlots; ++i) {
                at[i] = slot_hash(slot[i]);
                key[i] = sh.slot[at[i]];
            }
#pragma unroll
            for (int i = 0; i < kBatchSlots; ++i) {
                if (slot[i] < 0 || key[i] < 0) continue;     // most are not this CTA's
                const int place = slot_place(sh.slot, slot[i]);
                if (sh.slot[place] == slot[i]) atomicMax(&sh.token[place], t + i * kWarps * 32);
            }
        }
        __syncthreads();
    }

    Pairs a0, a1, b0 = {}, b1 = {};                          // A and B of this lane's chunks
    int32_t have_token = -1, have = -1;                      // what c, s and A, B are of
    for (int32_t i = 0; i < count; ++i) {
        ask(i + kAhead);
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
        __syncwarp();
        Stage& st = my.stage[i % kStages];
        const int32_t token = now.token;
        const Piece pc = piece_at(g, p, now.at);
        int32_t slot = -1;
        if constexpr (kStore) {
            slot = st.slot;
            if ((int64_t)slot >= g.num_slots) {
                if (lane == 0) pkv::report(g.status, PKV_STATUS_SLOT_OUT_OF_RANGE);
                slot = -1;
            }
            if (slot >= 0 && sh.token[slot_place(sh.slot, slot)] != token) slot = -1;
        }
        if (kStore && pc.which == 2) {                       // v rows, as they are
            if (slot >= 0) {
                uint4* to = (uint4*)(g.cache[1] + ((int64_t)slot * g.Hkv + pc.h0) * g.D);
                const int32_t vecs = pc.n * g.D * (int32_t)sizeof(T) / 16 - lane;
#pragma unroll
                for (int v = 0; v < kPieceBytes / 16; v += 32)
                    if (v < vecs) to[lane + v] = st.rows[lane + v];
            }
        } else {
            if (token != have_token) {
                have_token = token;
                have = -1;
                if constexpr (kPartner != kNone) {
                    const uint64_t pos = (uint64_t)(int64_t)st.position;
                    for (int t = lane; t < half; t += 32) {
                        float c, s;
                        turn(pos * __ldg((const unsigned long long*)g.turns + t), c, s);
                        my.c[t] = c * g.magnitude;
                        my.s[t] = s * g.magnitude;
                    }
                    __syncwarp();
                }
            }
            if (pc.which != have) {
                have = pc.which;
                const float* weight = sh.weight[pc.which];
                a0 = table_at(weight + e0);
                a1 = table_at(weight + e1);
                if constexpr (kPartner == kChunks) {
                    if (j < away) {
                        const Pairs c = table_at(my.c + e0), s = table_at(my.s + e0);
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            b0.v[t] = mul2(mul2(a1.v[t], s.v[t]), pk2(-1.f, -1.f));
                            b1.v[t] = mul2(a0.v[t], s.v[t]);
                            a0.v[t] = mul2(a0.v[t], c.v[t]);
                            a1.v[t] = mul2(a1.v[t], c.v[t]);
                        }
                    }
                } else if constexpr (kPartner == kPairs) {
                    auto chunk = [&](int e, Pairs& ta, Pairs& tb) {
                        const float4 c = *reinterpret_cast<const float4*>(my.c + e / 2);
                        const float4 s = *reinterpret_cast<const float4*>(my.s + e / 2);
                        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            if (e + 2 * t >= g.rotary_dim) break;
                            tb.v[t] = mul2(swapped(ta.v[t]), pk2(-ss[t], ss[t]));
                            ta.v[t] = mul2(ta.v[t], pk2(cc[t], cc[t]));
                        }
                    };
                    chunk(e0, a0, b0);
                    chunk(e1, a1, b1);
                } else if constexpr (kPartner == kShared) {
                    // A (from the weight) and B of entry e
                    auto entry = [&](int e, float& a, float& b) {
                        b = 0.f;
                        if (e >= g.rotary_dim) return;
                        const int t = e < half ? e : e - half;
                        a *= my.c[t];
                        b = e < half ? -weight[e + half] * my.s[t] : weight[t] * my.s[t];
                    };
                    auto quads = [&](int e, Pairs& ta, Pairs& tb) {
#pragma unroll
                        for (int t = 0; t < 4; t += 2, e += 4) {
                            tb.v[t] = tb.v[t + 1] = 0;
                            if (e >= g.rotary_dim) continue;
                            const bool second = e >= half;
                            const int at = second ? e - half : e;
                            const float sign = second ? 1.f : -1.f;
                            uint64_t c0, c1, s0, s1, o0, o1;
                            four(my.c + at, c0, c1);
                            four(my.s + at, s0, s1);
                            four(weight + (second ? at : e + half), o0, o1);
                            tb.v[t] = mul2(mul2(o0, pk2(sign, sign)), s0);
                            tb.v[t + 1] = mul2(mul2(o1, pk2(sign, sign)), s1);
                            ta.v[t] = mul2(ta.v[t], c0);
                            ta.v[t + 1] = mul2(ta.v[t + 1], c1);
                        }
                    };
                    auto chunk = [&](int e, Pairs& ta, Pairs& tb) {
                        if (half % 4 == 0) return quads(e, ta, tb);
#pragma unroll
                        for (int t = 0; t < 4; ++t, e += 2) {
                            float2 a = up2(ta.v[t]);
                            float b, d;
                            entry(e, a.x, b);
                            entry(e + 1, a.y, d);
                            ta.v[t] = pk2(a.x, a.y);
                            tb.v[t] = pk2(b, d);
                        }
                    };
                    chunk(e0, a0, b0);
                    chunk(e1, a1, b1);
                }
            }
            const bool norm = g.weight[pc.which] != nullptr;
            T* out = (T*)g.out[pc.which];
            if (out) out += token * g.out_stride[pc.which] + (int64_t)pc.h0 * g.D;
            T* cached = nullptr;
            if (kStore && pc.which == 1 && slot >= 0)
                cached = (T*)g.cache[0] + ((int64_t)slot * g.Hkv + pc.h0) * g.D;
            const T* rows = reinterpret_cast<const T*>(st.rows);
            // The piece's heads, and once more where there are some with squares beyond 32 bits.
            bool odd = false;
            auto heads = [&](auto scaled) {
                constexpr bool kScaled = decltype(scaled)::value;
#pragma unroll (kScaled ? 1 : 2)
                for (int32_t base = 0; base < pc.n; base += kHeads) {
                    // lanes without a head or a chunk compute on another's, and write nothing
                    const int32_t h = base + head < pc.n ? base + head : 0;
                    const bool in = base + head < pc.n && has0;
                    const T* row = rows + h * g.D;
                    Eight<T> x0, x1;
                    x0.take(row + e0);
                    x1.take(row + e1);
                    Pairs a = x0.get(), b = x1.get();
                    float r = 1.f, unit = 1.f;
                    if (norm) {
                        auto squares = [&] {
                            uint64_t s2 = mul2(a.v[0], a.v[0]);
#pragma unroll
                            for (int t = 1; t < 4; ++t) s2 = fma2(a.v[t], a.v[t], s2);
                            uint64_t both = s2;
#pragma unroll
                            for (int t = 0; t < 4; ++t) both = fma2(b.v[t], b.v[t], both);
                            const float2 s = up2(has1 ? both : s2);
                            float ss = has0 ? s.x + s.y : 0.f;
#pragma unroll
                            for (int off = kLanes / 2; off > 0; off >>= 1)
                                ss += __shfl_xor_sync(~0u, ss, off);
                            return ss;
                        };
                        float ss = squares(), eps = g.eps;
                        odd |= odd_squares(ss);
                        if constexpr (kScaled) {
                            if (odd_squares(ss)) unit = odd_unit(g, ss);
                            scale(a, unit);
                            scale(b, unit);
                            ss = squares();
                            eps = eps * unit * unit;
                        }
                        r = rsqrtf(fmaf(ss, g.inv_dim, eps));
                    }
                    const uint64_t r2 = pk2(r, r);
                    Pairs y0, y1;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        y0.v[t] = mul2(a0.v[t], a.v[t]);
                        y1.v[t] = mul2(a1.v[t], b.v[t]);
                    }
                    if constexpr (kPartner == kPairs) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            if (e0 + 2 * t < g.rotary_dim)
                                y0.v[t] = fma2(b0.v[t], swapped(a.v[t]), y0.v[t]);
                            if (e1 + 2 * t < g.rotary_dim)
                                y1.v[t] = fma2(b1.v[t], swapped(b.v[t]), y1.v[t]);
                        }
                    } else if constexpr (kPartner == kChunks) {
                        if (j < away) {
#pragma unroll
                            for (int t = 0; t < 4; ++t) {
                                y0.v[t] = fma2(b0.v[t], b.v[t], y0.v[t]);
                                y1.v[t] = fma2(b1.v[t], a.v[t], y1.v[t]);
                            }
                        }
                    } else if constexpr (kPartner == kShared) {
                        auto chunk = [&](int e, const Pairs& tb, Pairs& y) {
                            const uint64_t f2 = pk2(unit, unit);
                            if (half % 4 == 0) {
#pragma unroll
                                for (int t = 0; t < 4; t += 2, e += 4) {
                                    if (e >= g.rotary_dim) break;
                                    uint64_t lo, hi;
                                    four(row + (e < half ? e + half : e - half), lo, hi);
                                    if (kScaled) lo = mul2(lo, f2), hi = mul2(hi, f2);
                                    y.v[t] = fma2(tb.v[t], lo, y.v[t]);
                                    y.v[t + 1] = fma2(tb.v[t + 1], hi, y.v[t + 1]);
                                }
                            } else {
                                auto one = [&](int e) {
                                    return (float)row[e < half ? e + half : e - half];
                                };
#pragma unroll
                                for (int t = 0; t < 4; ++t, e += 2) {
                                    if (e >= g.rotary_dim) break;
                                    uint64_t x2 = pk2(one(e), one(e + 1));
                                    if (kScaled) x2 = mul2(x2, f2);
                                    y.v[t] = fma2(tb.v[t], x2, y.v[t]);
                                }
                            }
                        };
                        chunk(e0, b0, y0);
                        chunk(e1, b1, y1);
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        y0.v[t] = mul2(y0.v[t], r2);
                        y1.v[t] = mul2(y1.v[t], r2);
                    }
                    if (in && out) {
                        Eight<T>::store(out + h * g.D + e0, y0);
                        if (has1) Eight<T>::store(out + h * g.D + e1, y1);
                    }
                    if (kStore && in && cached) {
                        Eight<T>::store(cached + h * g.D + e0, y0);
                        if (has1) Eight<T>::store(cached + h * g.D + e1, y1);
                    }
                }
            };
            heads(std::false_type());
            if constexpr (kAnySquares<T>)
                if (__any_sync(~0u, odd)) heads(std::true_type());
        }
        __syncwarp();                                        // the stage is read
        advance(now);
    }
}

template <typename T, int kLanes, Partner kPartner, bool kStore>
int launch(const HeadArgs& g, cudaStream_t s) {
    if (g.num_tokens < kManyTokens) {
        head_kernel<T, kLanes, kPartner, kStore><<<(unsigned)g.num_tokens, kThreads, 0, s>>>(g);
    } else {
        static std::atomic<uint64_t> done{0};
        if (!pkv_dynamic_smem_once((const void*)row_kernel<T, kLanes, kPartner, kStore>,
                                   (int)sizeof(RowShared), done))
            return PKV_ERR_CUDA;
        constexpr int kHeads = 32 / kLanes;
        Pieces p;
        p.heads = kPieceBytes / (g.D * (int)sizeof(T)) / kHeads * kHeads;
        p.of_q = (g.Hq + p.heads - 1) / p.heads;
        p.of_k = (g.Hkv + p.heads - 1) / p.heads;
        p.per_token = p.of_q + p.of_k * (kStore ? 2 : 1);
        // as many tokens a launch as the table of slots has room for: later launches, with
        // later tokens, write later
        const int32_t room = pkv_num_sms() * (kStore ? kTokensPerCta : 1 << 22);
        HeadArgs part = g;
        for (int32_t from = 0; from < g.num_tokens;) {
            part.num_tokens = g.num_tokens - from < room ? g.num_tokens - from : room;
            const int64_t units = (int64_t)p.per_token * part.num_tokens;
            int64_t grid = (units + kWarps - 1) / kWarps;
            if (grid > pkv_num_sms()) grid = pkv_num_sms();
            row_kernel<T, kLanes, kPartner, kStore>
                <<<(unsigned)grid, kWarps * 32, sizeof(RowShared), s>>>(part, p);
            from += part.num_tokens;
            for (int i = 0; i < 3; ++i)
                if (g.in[i])
                    part.in[i] = (const T*)g.in[i] + (int64_t)from * g.in_stride[i];
            for (int i = 0; i < 2; ++i)
                if (g.out[i]) part.out[i] = (T*)g.out[i] + (int64_t)from * g.out_stride[i];
            if (g.positions) part.positions = g.positions + from;
            if (g.slots) part.slots = g.slots + from;
        }
    }
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

template <typename T, int kLanes, bool kStore>
int launch(const HeadArgs& g, cudaStream_t s) {
    return g.rotary_dim == 0        ? launch<T, kLanes, kNone, kStore>(g, s)
           : g.interleaved          ? launch<T, kLanes, kPairs, kStore>(g, s)
           : g.rotary_dim % 16 == 0 ? launch<T, kLanes, kChunks, kStore>(g, s)
                                    : launch<T, kLanes, kShared, kStore>(g, s);
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
    // eps tiny_unit^2 at most 2^120
    int e = -126;
    if (eps > 0.f) frexpf(eps, &e);
    g.tiny_unit = ldexpf(1.f, e < -80 ? 100 : (120 - e) / 2);
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
