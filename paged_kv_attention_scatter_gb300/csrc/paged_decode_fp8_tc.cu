// paged_decode_fp8 split kernel on the 5th-generation tensor cores, for any block
// size and head_dim 128 or 64.
//
// The sums are those stated in paged_decode_fp8.cu.  Here the codes are never
// converted: tcgen05.mma takes them as they lie in shared memory, keys (for S)
// and head_dim (for O) as its 128 rows, and the at most 8 q heads of a unit as
// its 16 columns:
//   S[key, n] = K8[key, :] . Q[n, :]      A = K, K-major;   B = Q, K-major
//   O[d, n]   = sum_key V8[key, d] P[key, n]   A = V, MN-major;  B = P, MN-major
// Q and P have to be e4m3 as well, whose significand is 4 bits; each is the sum
// of two e4m3 values, in a column of its own each, H columns apart:
//   q * up = q1 + q2 / 16, up the power of two that brings a row's largest entry
//     to [2^7, 2^8).  A bf16 has 8 significant bits, so q1 rounds to the first 4
//     and q2 holds the rest exactly, down to 2^-22 of the row's largest entry.
//   p = 2^(y - M + 8) <= 256 likewise: off by 2^-9 of itself, or 2^-22 of the
//     row's largest weight.  (Scores past 2^20 have a step of their own of 2^-3 and
//     more; M may be rounded up there by up to 12, and p smaller by as much.)
// M is the running maximum over all keys of the unit that a softmax group has seen: its four
// warps exchange their maxima each stage, so no p exceeds 256.  (A reference that
// lags, redone when it is passed, needs headroom that e4m3 lacks: 448 / 256.)
//
// Roles, one CTA per SM, a ring of 128-key stages (32 KB):
//   warps 0-7  softmax, two groups of four that take a CTA's stages in turn (a
//              stage's chain of steps is longer than its bytes take to arrive).
//              Thread i of a group has key i of a stage (TMEM lane i).  It reads
//              the key's S columns, exchanges maxima, writes the key's 16 bytes of
//              P (one 16-byte store: B, MN-major, 16 columns wide) and zeroes the V
//              row of a key that does not count (0 * NaN is NaN).  Then it takes the
//              O of its group's stage before, thread i being head_dim entry i now,
//              and adds it to fp32 registers: O = (O + O') alpha.  TMEM accumulates
//              within a stage only, so nothing in it is ever rescaled.  The group
//              with a unit's last stage merges the other's share and writes it.
//   warp 8     S issuer, up to three stages ahead of the softmax (two S buffers a
//              group).
//   warp 9     P V issuer; its completion frees the stage's slot.
//   warp 10    Q: scales, splits and lays out the next units' rows.
//   warp 11    producer, block sizes that are multiples of 64: per stage two
//              (head_dim 64: four) 64-key TMA boxes of K and as many of V, each in one
//              cache block, with its scales in the stage's record.
//   warps 11-18 producers, other block sizes, four teams of two that fill stages
//              in turn: a lane looks up its keys' blocks and scales, the warp
//              gathers half a stage's rows with 16-byte cp.async into the layout the boxes
//              would have; rows that do not count are filled with zeros.
// Every mbarrier wait is bounded; on expiry the CTA unwinds as in
// paged_decode_tma.cu, and TMEM is freed after its last MMA.
//
// An mma.sync kernel with the same stages (codes converted to f16, two thirds of
// each MMA idle, the warps' partial outputs merged per unit) took 91 and 265 us
// where this one takes 54 and 190 (64 sequences of 16/8 heads, 512..4096 keys; 96
// of 64/8 heads, 128..32768 keys, block size 256), and one loading registers
// straight from the cache 179 us where this one takes 74 (48 of 32/8 heads,
// 1..8192 keys, block size 16).
#include <cudaTypedefs.h>

#include "fp8_common.cuh"
#include "tc_utils.cuh"
#include "tma_host.cuh"

using pkv::Fp8DecodeArgs;
using pkv::kMaxGroup;

namespace {

namespace tc = pkv::tc;

constexpr int kBoxKeys = 64;
constexpr int kCols = 16;                        // MMA N
constexpr int kGroups = 2, kGroupWarps = 4;     // softmax groups of 128 threads
constexpr int kSWarp = kGroups * kGroupWarps, kPvWarp = kSWarp + 1, kQWarp = kSWarp + 2;
constexpr int kFirstProducer = kSWarp + 3;
constexpr int kBufs = 2 * kGroups;               // S, P and O buffers: two a group
constexpr int kQPow = 8;                         // a power of two; see the Q role
constexpr int kTeams = 4, kTeamWarps = 2;        // gathering warps: a team fills a stage
constexpr int kGatherWarps = kTeams * kTeamWarps;

struct alignas(16) StageMeta {
    int32_t j, n;                                // stage j of the unit's n; n 0: no more stages
    int32_t keys;                                // from the stage's first to the chunk's end
    int32_t unit;                                // of this CTA, counted up
    int32_t row, h0, nh, nch;                    // row: of part_o, or of out if nch is 1
};

template <int D>
struct Smem {
    // a stage is 32 KB, K and V: 128 keys, or 256 of head_dim 64 (two a thread, so
    // that a stage's fixed costs are spread over as many bytes)
    static constexpr int kTileBytes = 128 * 128;
    static constexpr int kStageKeys = kTileBytes / D;
    static constexpr int kStages = D == 128 ? 6 : 5;
    uint8_t kv[kStages][2 * kTileBytes];         // K tile, V tile; 1024-byte aligned
    alignas(1024) uint8_t q[2][kCols * D];       // by unit parity, swizzled
    alignas(16) uint8_t p[kBufs][kStageKeys * kCols];
    float ks[kStages][kStageKeys];               // per key (gathered) or box: K scale,
    float lv[kStages][kStageKeys];               // log2 of V's (-inf: does not count),
    float rv[kStages][kStageKeys];               // 1 / (4 sqrt(V's))
    StageMeta meta[kStages];
    alignas(16) float q_pow[kQPow][kMaxGroup];
    alignas(16) float warp_ref[kBufs][kGroupWarps][kMaxGroup];
    alignas(16) float warp_sum[kGroups][2][kMaxGroup][kGroupWarps];
    // one group's share of a unit, for the group that finishes it
    alignas(16) float ex_o[kMaxGroup][D];
    alignas(16) float ex_l[kMaxGroup][kGroupWarps];
    alignas(16) float ex_c[kMaxGroup];
    uint64_t full[kStages], empty[kStages];
    uint64_t s_full[kBufs], p_full[kBufs], o_full[kBufs];
    uint64_t q_full[2], q_empty[2];
    uint64_t max_bar[kGroups], sum_bar[kGroups], ex_full, ex_free, drain_s, drain_o;
    uint32_t tmem;
    int abort_flag;
};

static_assert(sizeof(Smem<128>) + 1024 <= 232448 && sizeof(Smem<64>) + 1024 <= 232448,
              "more shared memory than a CTA can have");

// Instruction descriptor of tcgen05.mma.kind::f8f6f4: e4m3 A and B (both K-major
// or both MN-major), fp32 D, rows x 16.
__host__ __device__ constexpr uint32_t idesc_e4m3(bool mn_major, int rows) {
    return (1u << 4) | ((mn_major ? 3u : 0u) << 15) | ((uint32_t)(kCols >> 3) << 17) |
           ((uint32_t)(rows >> 4) << 24);
}

// Descriptor of rows of D bytes in D-byte swizzle atoms of 8 rows: K and Q
// (K-major) and V (MN-major, one atom wide): the stride from 8 rows to the next 8.
template <int D>
__device__ __forceinline__ uint64_t rows_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 |
           (uint64_t)((8 * D) >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)(D == 128 ? 2 : 4) << 61;
}

// Byte offset of 16-byte chunk c of row r in that layout (64-byte swizzle: two
// rows a 128-byte line, chunk ^ line).
template <int D>
__device__ __forceinline__ int swz(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Descriptor of P: MN-major without swizzle.  A core matrix is 8 keys of 16
// columns (16 bytes), and the operand is one core matrix wide, so the only
// stride is the one along the keys, 128 bytes.
__device__ __forceinline__ uint64_t p_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 16 |
           (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// N consecutive fp32 columns of this thread's TMEM lane; there after tmem_wait_ld.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float* v) {
    if constexpr (N == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                     : "r"(addr));
    } else if constexpr (N == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                       "=f"(v[6]), "=f"(v[7])
                     : "r"(addr));
    } else {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
              "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
              "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
            : "r"(addr));
    }
}
// Waits for this thread's tcgen05.ld; the values pass through it, so that no use
// of them moves ahead of the wait.
template <int N>
__device__ __forceinline__ void tmem_wait(float* v) {
    tc::tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
          "l"(reinterpret_cast<uint64_t&>(c)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t&>(d))
        : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
    return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// A factor in fp32's range, NaN if it is NaN.
__device__ __forceinline__ float saturate(float x) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(3.4028234663852886e38f));
    return r;
}

// 6 - m / 2 rounded down, so that m / 2 and it add up to at most 6 (and at least 0, as
// -m / 2 is a number itself): the reference of weights whose largest score is m.  +inf
// for a maximum over nothing.
__device__ __forceinline__ float half_ref(float m) { return __fmaf_rd(m, -0.5f, 6.f); }

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(uint32_t x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
    return r;
}

// x16 = 16 x (f16x2, |x| <= 256) as x = hi + lo / 16, both pairs of e4m3: the
// first four significant bits and what they leave, which 16 x - 16 hi gives
// exactly.
__device__ __forceinline__ void split_e4m3(uint32_t x16, uint16_t& hi, uint16_t& lo) {
    hi = f16x2_to_e4m3x2(mul_f16x2(x16, 0x2c002c00u));                     // 1/16
    lo = f16x2_to_e4m3x2(fma_f16x2(pkv::e4m3x2_to_f16x2(hi), 0xcc00cc00u, x16));  // -16
}

__device__ __forceinline__ void cp_async16(void* smem, const void* gmem, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::saddr(smem)),
                 "l"(gmem), "r"(bytes)
                 : "memory");
}

// The chunk records, as a warp reads them: from the plan kernel's list, or from
// the warp's own plan.
struct Schedule {
    pkv::WarpPlan plan;
    const int4* records;
    int32_t chunks, chunk_keys;
    bool own;
    __device__ __forceinline__ explicit Schedule(const pkv::DecodeArgs& a)
        : plan(own_args(a)), records(a.chunk_info), chunk_keys(a.chunk_keys),
          own(a.inline_plan != 0) {
        chunks = own ? plan.total() : a.chunk_prefix[a.B];
    }
    // (a plan of no sequences where the list is used)
    __device__ __forceinline__ static pkv::DecodeArgs own_args(const pkv::DecodeArgs& a) {
        pkv::DecodeArgs x = a;
        if (!a.inline_plan) x.B = 0;
        return x;
    }
    // no keys past the last chunk
    __device__ __forceinline__ int4 record(int32_t sc) const {
        if (sc >= chunks) return make_int4(0, 0, 0, 0);
        return own ? plan.record(sc, chunk_keys) : records[sc];
    }
};

// A CTA's units in order: unit u is (chunk u / per_sc, kv head, group of q
// heads).  The CTA takes u = blockIdx.x, + gridDim.x, ...; a step is an addition
// with carry, not a division.
struct Units {
    int32_t sc, rem, per_sc, n_hg, step_sc, step_rem;
    __device__ __forceinline__ explicit Units(const pkv::DecodeArgs& a) {
        per_sc = a.Hkv * a.n_hg;
        n_hg = a.n_hg;
        sc = (int32_t)blockIdx.x / per_sc;
        rem = (int32_t)blockIdx.x % per_sc;
        step_sc = (int32_t)gridDim.x / per_sc;
        step_rem = (int32_t)gridDim.x % per_sc;
    }
    __device__ __forceinline__ void next() {
        sc += step_sc;
        rem += step_rem;
        if (rem >= per_sc) {
            rem -= per_sc;
            ++sc;
        }
    }
    __device__ __forceinline__ int32_t kv_head() const { return n_hg == 1 ? rem : rem / n_hg; }
    __device__ __forceinline__ int32_t head_group() const { return n_hg == 1 ? 0 : rem % n_hg; }
};

// A ring position that several roles walk alike.
template <int kStages>
struct RingOf {
    int slot = 0;
    uint32_t phase = 0, laps = 0;
    __device__ __forceinline__ void next(int by = 1) {
        slot += by;
        if (slot >= kStages) {
            slot -= kStages;
            phase ^= 1;
            ++laps;
        }
    }
};

// kHeads: q heads a unit may have (2, 4 or 8).  kGather: any block size.
template <int D, int kHeads, bool kGather, bool kPolls>
__global__ void __launch_bounds__((kFirstProducer + (kGather ? kGatherWarps : 1)) * 32, 1)
    decode_fp8_tc_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, Fp8DecodeArgs fa) {
    const pkv::DecodeArgs& a = fa.d;
    const uint32_t polls = kPolls ? a.wait_polls : (uint32_t)PKV_DEFAULT_WAIT_POLLS;
    using Sm = Smem<D>;
    constexpr int kStages = Sm::kStages, kTileBytes = Sm::kTileBytes, kStageKeys = Sm::kStageKeys;
    constexpr int kSub = kStageKeys / 128;       // keys of a stage per softmax thread
    constexpr int kBoxes = kStageKeys / kBoxKeys;
    constexpr int kTmemO = kBufs * kSub * kCols; // columns: the S buffers, then the O buffers
    constexpr int kTmemCols = D == 128 ? 128 : 256;
    constexpr int kGatherRows = kStageKeys / kTeamWarps;         // rows of a stage per warp
    using Ring = RingOf<kStages>;
    extern __shared__ uint8_t smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&sm.full[s], kGather ? kTeamWarps : 1);
            tc::mbar_init(&sm.empty[s], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            tc::mbar_init(&sm.s_full[i], 1);
            tc::mbar_init(&sm.p_full[i], kGroupWarps);
            tc::mbar_init(&sm.o_full[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sm.q_full[i], 1);
            tc::mbar_init(&sm.q_empty[i], 1);
            tc::mbar_init(&sm.max_bar[i], kGroupWarps);
            tc::mbar_init(&sm.sum_bar[i], kGroupWarps);
        }
        tc::mbar_init(&sm.ex_full, kGroupWarps);
        tc::mbar_init(&sm.ex_free, kGroupWarps);
        tc::mbar_init(&sm.drain_s, 1);
        tc::mbar_init(&sm.drain_o, 1);
        sm.abort_flag = 0;
        tc::mbar_init_fence();
    }
    // the Q rows that no head fills, once
    for (int i = threadIdx.x; i < (int)sizeof(sm.q) / 16; i += blockDim.x)
        reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0, 0, 0, 0);
    if (warp == kSWarp) tc::tmem_alloc(&sm.tmem, kTmemCols);
    tc::fence_proxy_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = sm.tmem;
    pkv::wait_for_predecessor();                 // the plan kernel's chunk records
    pkv::allow_dependent_launch();

    auto give_up = [&]() {
        *(volatile int*)&sm.abort_flag = 1;
        pkv::report(a.status, PKV_STATUS_WAIT_TIMEOUT);
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return tc::mbar_wait(bar, parity, &sm.abort_flag, polls);
    };
    // the same for a whole warp: one outcome for all its lanes
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };

    if (warp < kSWarp) {
        // ------------------------------------------------------------- softmax
        const int group = warp / kGroupWarps, gw = warp % kGroupWarps;
        const uint32_t lane_base = tmem + ((uint32_t)(gw * 32) << 16);
        // thread i of the group: keys i (and i + 128) of a stage, TMEM lane i; and the
        // head_dim entry of O in that lane: 128 rows are the lanes, 64 rows the
        // first 16 of each warp's
        const int key = threadIdx.x % 128;
        const int dim = D == 128 ? key : lane < 16 ? gw * 16 + lane : -1;
        Ring ring;
        ring.next(group);
        uint32_t shared = 0, units = 0;          // units of both groups; units of this one
        float c_run[kHeads], l[kHeads], o[kHeads], xs[kHeads];       // c_run: half_ref(M)
#pragma unroll
        for (int h = 0; h < kHeads; ++h) c_run[h] = l[h] = o[h] = xs[h] = 0.f;
        bool ok = true;
        for (uint32_t c = 0;; ++c, ring.next(kGroups)) {     // this group's stages
            const int buf = 2 * group + (c & 1), before = 2 * group + ((c & 1) ^ 1);
            const uint32_t par = (c >> 1) & 1;
            if (!(ok = wait_warp(&sm.full[ring.slot], ring.phase))) break;
            const StageMeta meta = sm.meta[ring.slot];
            if (meta.n == 0) break;
            const bool first = meta.j < kGroups, last = meta.j + kGroups >= meta.n;
            float ks[kSub], lv[kSub], rv[kSub];
            bool counts[kSub];
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                const int mine = kGather ? key + 128 * u : (key + 128 * u) / kBoxKeys;
                ks[u] = sm.ks[ring.slot][mine];
                lv[u] = sm.lv[ring.slot][mine];
                rv[u] = sm.rv[ring.slot][mine];
                counts[u] = lv[u] != -INFINITY && (kGather || key + 128 * u < meta.keys);
            }
            if (!(ok = wait_warp(&sm.s_full[buf], par))) break;
            tc::tc_fence_after();
            float s[kSub][2 * kHeads], y[kSub][kHeads];
#pragma unroll
            for (int u = 0; u < kSub; ++u)
                tmem_ld<2 * kHeads>(lane_base + (buf * kSub + u) * kCols, s[u]);
            tmem_wait<kSub * 2 * kHeads>(&s[0][0]);
            if (first) {                         // (the S issuer has waited for Q)
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    xs[h] = fabsf(a.scale_log2) * sm.q_pow[meta.unit % kQPow][h];
                    c_run[h] = INFINITY;
                    l[h] = o[h] = 0.f;
                }
            }
            // y = dot ks xs + lv, the heads two by two; -inf where the key does not
            // count, whose dot may be anything.  The factor saturates, so that a dot
            // of zero beside it stays zero (any other is a score past 2^100 then).
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
#pragma unroll
                for (int h = 0; h < kHeads; h += 2) {
                    const float2 dot = fma2(make_float2(s[u][kHeads + h], s[u][kHeads + h + 1]),
                                            both(0.0625f), make_float2(s[u][h], s[u][h + 1]));
                    float2 k = mul2(both(ks[u]), make_float2(xs[h], xs[h + 1]));
                    k = make_float2(saturate(k.x), saturate(k.y));
                    const float2 x = fma2(dot, k, both(lv[u]));
                    y[u][h] = x.x;
                    y[u][h + 1] = x.y;
                }
                if (!__all_sync(0xffffffffu, counts[u])) {
#pragma unroll
                    for (int h = 0; h < kHeads; ++h)
                        if (!counts[u]) y[u][h] = -INFINITY;
                }
            }
            // ---- the stage's maxima, as half references (half_ref falls with its argument) ----
            float top[kHeads];
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                top[h] = y[0][h];
                if constexpr (kSub == 2) top[h] = fmaxf(top[h], y[1][h]);
                top[h] = half_ref(warp_max(top[h]));
            }
            if (lane == 0) {
#pragma unroll
                for (int h = 0; h < kHeads; h += 2)
                    *reinterpret_cast<float2*>(&sm.warp_ref[buf][gw][h]) =
                        make_float2(top[h], top[h + 1]);
                tc::mbar_arrive(&sm.max_bar[group]);
            }
            if (!(ok = wait_warp(&sm.max_bar[group], c & 1))) break;
            float alpha[kHeads], use[kHeads];
#pragma unroll
            for (int h = 0; h < kHeads; ++h) use[h] = c_run[h];
#pragma unroll
            for (int w = 0; w < kGroupWarps; ++w) {
                if constexpr (kHeads == 2) {
                    const float2 x = *reinterpret_cast<const float2*>(sm.warp_ref[buf][w]);
                    use[0] = fminf(use[0], x.x);
                    use[1] = fminf(use[1], x.y);
                } else {
#pragma unroll
                    for (int h = 0; h < kHeads; h += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(&sm.warp_ref[buf][w][h]);
                        use[h] = fminf(use[h], x.x);
                        use[h + 1] = fminf(use[h + 1], x.y);
                        use[h + 2] = fminf(use[h + 2], x.z);
                        use[h + 3] = fminf(use[h + 3], x.w);
                    }
                }
            }
            // Weights by their square roots, against c = 6 - M / 2 rounded down (half_ref):
            // g = 2^(y / 2 + c) is at most 2^6 and normal down to 2^-264 of the largest
            // weight.  16 p = g^2, and l's term is (g rv)^2 = 256 / vs of the weight, so a
            // key counts there however small its V scale is beside the largest (its p
            // may vanish: that is its share of O).  Every step and merge takes the
            // difference of two c, so what their rounding leaves out cancels.
#pragma unroll
            for (int h = 0; h < kHeads; h += 2) {
                const float2 c2 = make_float2(use[h] == INFINITY ? 6.f : use[h],
                                              use[h + 1] == INFINITY ? 6.f : use[h + 1]);
                const float2 a2 = make_float2(pkv::fast_exp2(c2.x - c_run[h]),       // 0 from +inf
                                              pkv::fast_exp2(c2.y - c_run[h + 1]));
                const float2 squared = mul2(a2, a2);
                float2 sum = mul2(mul2(make_float2(l[h], l[h + 1]), a2), a2);
                alpha[h] = squared.x;
                alpha[h + 1] = squared.y;
                c_run[h] = use[h];
                c_run[h + 1] = use[h + 1];
#pragma unroll
                for (int x = 0; x < kSub; ++x) {
                    const float2 e = fma2(make_float2(y[x][h], y[x][h + 1]), both(0.5f), c2);
                    const float2 g = make_float2(pkv::fast_exp2(e.x), pkv::fast_exp2(e.y));
                    const float2 t = mul2(g, both(rv[x]));
                    sum = fma2(t, t, sum);
                    const float2 p16 = mul2(g, g);           // as split_e4m3 takes it
                    y[x][h] = p16.x;
                    y[x][h + 1] = p16.y;
                }
                l[h] = sum.x;
                l[h + 1] = sum.y;
            }
            // ---- the keys' rows of P: bytes h the first parts, kHeads + h the second ----
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int h = 0; h < kHeads; h += 2) {
                    uint16_t hi, lo;
                    split_e4m3(pkv::pack_f16(y[u][h], y[u][h + 1]), hi, lo);
                    w[h / 4] |= (uint32_t)hi << (h % 4 * 8);
                    w[(kHeads + h) / 4] |= (uint32_t)lo << ((kHeads + h) % 4 * 8);
                }
                *reinterpret_cast<uint4*>(sm.p[buf] + (key + 128 * u) * kCols) =
                    make_uint4(w[0], w[1], w[2], w[3]);
                if (!counts[u]) {
                    uint4* v = reinterpret_cast<uint4*>(sm.kv[ring.slot] + kTileBytes +
                                                        (key + 128 * u) * D);
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) v[i] = make_uint4(0, 0, 0, 0);
                }
            }
            tc::fence_proxy_async_smem();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm.p_full[buf]);
            // ---- the O of the group's stage before, and at a unit's end this one's ----
            float t[2 * kHeads];
            if (!first) {
                if (!(ok = wait_warp(&sm.o_full[before], ((c - 1) >> 1) & 1))) break;
                tc::tc_fence_after();
                tmem_ld<2 * kHeads>(lane_base + kTmemO + before * kCols, t);
                tmem_wait<2 * kHeads>(t);
#pragma unroll
                for (int h = 0; h < kHeads; h += 2) {
                    const float2 x = fma2(make_float2(t[kHeads + h], t[kHeads + h + 1]),
                                          both(0.0625f), make_float2(t[h], t[h + 1]));
                    const float2 sum = mul2(add2(make_float2(o[h], o[h + 1]), x),
                                            make_float2(alpha[h], alpha[h + 1]));
                    o[h] = sum.x;
                    o[h + 1] = sum.y;
                }
            }
            if (!last) continue;
            // the warp's sums, while the last P V runs: a lane passes on half of its heads
            // at a step and ends with the sum of head lane / (32 / kHeads)
#pragma unroll
            for (int left = kHeads / 2, off = 16; off > 0; left >>= 1, off >>= 1) {
                if (left > 0) {
                    const bool upper = lane & off;
#pragma unroll
                    for (int h = 0; h < left; ++h) {
                        const float give = upper ? l[h] : l[left + h];
                        const float keep = upper ? l[left + h] : l[h];
                        l[h] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                    }
                } else {
                    l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
                }
            }
            const int l_head = lane / (32 / kHeads);
            const bool l_mine = lane % (32 / kHeads) == 0;
            if (!(ok = wait_warp(&sm.o_full[buf], par))) break;
            tc::tc_fence_after();
            tmem_ld<2 * kHeads>(lane_base + kTmemO + buf * kCols, t);
            tmem_wait<2 * kHeads>(t);
#pragma unroll
            for (int h = 0; h < kHeads; ++h) o[h] += fmaf(t[kHeads + h], 0.0625f, t[h]);
            if (meta.j + 1 < meta.n) {
                // the other group has the unit's last stage: hand this share over
                // once the share before has been read
                if (shared > 0 && !(ok = wait_warp(&sm.ex_free, (shared - 1) & 1))) break;
                ++shared;
#pragma unroll
                for (int h = 0; h < kHeads; ++h) {
                    if (dim >= 0) sm.ex_o[h][dim] = o[h];
                    if (key == 0) sm.ex_c[h] = c_run[h];
                }
                if (l_mine) sm.ex_l[l_head][gw] = l[0];
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sm.ex_full);
                continue;
            }
            float (*sums)[kGroupWarps] = sm.warp_sum[group][units & 1];
            if (l_mine) sums[l_head][gw] = l[0];
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm.sum_bar[group]);
            if (!(ok = wait_warp(&sm.sum_bar[group], units & 1))) break;
            ++units;
            const bool both = meta.n > 1;
            if (both && !(ok = wait_warp(&sm.ex_full, shared & 1))) break;
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                const float4 mine = *reinterpret_cast<const float4*>(sums[h]);
                float L = (mine.x + mine.y) + (mine.z + mine.w), O = o[h], c1 = c_run[h];
                if (both) {
                    const float4 other = *reinterpret_cast<const float4*>(sm.ex_l[h]);
                    const float L2 = (other.x + other.y) + (other.z + other.w);
                    const float c2 = sm.ex_c[h], cm = fminf(c1, c2);
                    const float to = cm == INFINITY ? 0.f : cm;
                    const float f1 = pkv::fast_exp2(to - c1), f2 = pkv::fast_exp2(to - c2);
                    L = fmaf(L * f1, f1, L2 * f2 * f2);
                    if (dim >= 0) O = fmaf(O, f1 * f1, sm.ex_o[h][dim] * (f2 * f2));
                    c1 = cm;
                }
                if (h >= meta.nh || dim < 0) continue;
                const int64_t at = (int64_t)meta.row + meta.h0 + h;
                if (meta.nch == 1) {
                    a.out[at * D + dim] = __float2bfloat16_rn(L == 0.f ? 0.f : O / L);
                } else {
                    a.part_o[at * D + dim] = O;
                    if (dim == 0) a.part_ml[at] = make_float2(-c1, L);         // M / 2 - 6, see the combine
                }
            }
            if (both) {
                ++shared;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sm.ex_free);
            }
        }
        if (!ok) give_up();
    } else if (warp == kSWarp) {
        // ------------------------------------------------------------ S issuer
        if (lane == 0) {
            Ring ring;
            bool ok = true;
            for (uint32_t it = 0;; ++it, ring.next()) {
                const uint32_t c = it / kGroups;             // of the stage's group
                const uint32_t buf = 2 * (it % kGroups) + (c & 1);
                if (!(ok = wait(&sm.full[ring.slot], ring.phase))) break;
                const int32_t j = sm.meta[ring.slot].j, n = sm.meta[ring.slot].n;
                const uint32_t unit = sm.meta[ring.slot].unit;
                if (n == 0) break;
                // the buffer's last S is read once its P is written
                if (c >= 2 && !(ok = wait(&sm.p_full[buf], ((c - 2) >> 1) & 1))) break;
                if (j == 0 && !(ok = wait(&sm.q_full[unit & 1], (unit >> 1) & 1))) break;
                tc::tc_fence_after();
                const uint64_t qd = rows_desc<D>(tc::saddr(sm.q[unit & 1]));
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
                    const uint64_t kd = rows_desc<D>(tc::saddr(sm.kv[ring.slot]) + u * 128 * D);
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)         // 32 codes = 32 bytes a step
                        mma_e4m3(tmem + (buf * kSub + u) * kCols, kd + k * 2, qd + k * 2,
                                 idesc_e4m3(false, 128), k > 0);
                }
                tc::umma_commit(&sm.s_full[buf]);
                if (j + 1 == n) tc::umma_commit(&sm.q_empty[unit & 1]);
            }
            if (!ok) give_up();
            tc::umma_commit(&sm.drain_s);                    // every MMA issued here is done
            tc::mbar_drain(&sm.drain_s, 0);
        }
    } else if (warp == kPvWarp) {
        // ---------------------------------------------------------- P V issuer
        if (lane == 0) {
            Ring ring;
            bool ok = true;
            for (uint32_t it = 0;; ++it, ring.next()) {
                const uint32_t c = it / kGroups;
                const uint32_t buf = 2 * (it % kGroups) + (c & 1);
                if (!(ok = wait(&sm.full[ring.slot], ring.phase))) break;
                if (sm.meta[ring.slot].n == 0) break;
                if (!(ok = wait(&sm.p_full[buf], (c >> 1) & 1))) break;
                tc::tc_fence_after();
                const uint64_t vd = rows_desc<D>(tc::saddr(sm.kv[ring.slot]) + kTileBytes);
                const uint64_t pd = p_desc(tc::saddr(sm.p[buf]));
#pragma unroll
                for (int k = 0; k < kStageKeys / 32; ++k)    // 32 keys a step
                    mma_e4m3(tmem + kTmemO + buf * kCols, vd + k * (32 * D >> 4),
                             pd + k * (32 * kCols >> 4),
                             idesc_e4m3(true, D), k > 0);
                tc::umma_commit(&sm.empty[ring.slot]);
                tc::umma_commit(&sm.o_full[buf]);
            }
            if (!ok) give_up();
            tc::umma_commit(&sm.drain_o);
            tc::mbar_drain(&sm.drain_o, 0);
        }
    } else if (warp == kQWarp) {
        // ------------------------------------------------------------------- Q
        // lane l: quarter l % 4 of head l / 4.  The operand has two
        // buffers, freed by the unit's last S.  The powers are read by the softmax,
        // up to three stages behind the S issuer and so up to three units; this
        // role is up to two units ahead of it: 8 buffers are enough.
        const int h = lane >> 2, part = lane & 3;
        const Schedule sched(a);
        if (sched.own && blockIdx.x == 0 && sched.plan.bad)
            pkv::report(a.status, PKV_STATUS_BAD_CONTEXT_LEN);
        if (fa.no_combine) {                     // the rows of sequences without keys
            for (int32_t b = blockIdx.x; b < a.B; b += gridDim.x) {
                const int32_t n = sched.own ? sched.plan.of(b).y
                                            : a.chunk_prefix[b + 1] - a.chunk_prefix[b];
                if (n > 0) continue;
                uint4* row = reinterpret_cast<uint4*>(a.out + (int64_t)b * a.Hq * D);
                for (int32_t i = lane; i < a.Hq * (D / 8); i += 32) row[i] = make_uint4(0, 0, 0, 0);
            }
        }
        Units un(a);
        uint32_t units = 0;
        bool ok = true;
        int32_t sequence = sched.record(un.sc).x;        // of the unit after: loaded a unit ahead
        for (; un.sc < sched.chunks; ++units) {
            const int32_t hg = un.head_group(), kvh = un.kv_head();
            const int32_t b = sequence;
            un.next();
            sequence = sched.record(un.sc).x;
            const int32_t h0 = kvh * a.G + hg * kMaxGroup;
            const bool there = h < kHeads && h < min(kMaxGroup, a.G - hg * kMaxGroup);
            constexpr int kChunks = D / 64;      // 16-entry chunks of the quarter
            uint4 raw[2 * kChunks];
#pragma unroll
            for (int i = 0; i < 2 * kChunks; ++i) {
                raw[i] = make_uint4(0, 0, 0, 0);
                if (there)
                    raw[i] = __ldg(reinterpret_cast<const uint4*>(
                                       a.q + ((int64_t)b * a.Hq + h0 + h) * D + part * (D / 4)) +
                                   i);
            }
            uint32_t mag = 0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint32_t x = pkv::word(raw[i >> 2], i & 3);
                const uint32_t lo = x & 0x7fffu, hi = (x >> 16) & 0x7fffu;
                mag = max(mag, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            }
            mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
            mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
            // an infinite entry makes the head's weights NaN; e4m3 has no infinity, so
            // it goes in as NaN.  A negative softmax scale's sign goes with q.
            auto no_inf = [&](uint32_t x) {
                x ^= a.scale_log2 < 0.f ? 0x80008000u : 0u;
                if ((x & 0x7fffu) == 0x7f80u) x |= 0x40u;
                if ((x & 0x7fff0000u) == 0x7f800000u) x |= 0x400000u;
                return x;
            };
            // largest entry 1.f * 2^(E - 127) to 1.f * 2^7: e >= -120, as E <= 254.  At
            // most 2^120, so that 16 times it and its inverse are normal fp32 numbers:
            // rows below 2^-113 stay below 2^7, but 2^120 takes bf16's smallest step,
            // 2^-133, to the second part's, 2^-13, so they are held exactly too.
            const int e = min(7 - ((int)(mag >> 7) - 127), 120);
            const float up16 = __int_as_float((e + 4 + 127) << 23);
            uint32_t hi[4 * kChunks], lo[4 * kChunks];       // the codes of either part
#pragma unroll
            for (int i = 0; i < D / 8; i += 2) {
                uint16_t a0, b0, a1, b1;
                const uint32_t x = no_inf(pkv::word(raw[i >> 2], i & 3));
                const uint32_t z = no_inf(pkv::word(raw[i >> 2], (i & 3) + 1));
                split_e4m3(pkv::pack_f16(__int_as_float((int)(x << 16)) * up16,
                                         __int_as_float((int)(x & 0xffff0000u)) * up16),
                           a0, b0);
                split_e4m3(pkv::pack_f16(__int_as_float((int)(z << 16)) * up16,
                                         __int_as_float((int)(z & 0xffff0000u)) * up16),
                           a1, b1);
                hi[i >> 1] = (uint32_t)a0 | (uint32_t)a1 << 16;
                lo[i >> 1] = (uint32_t)b0 | (uint32_t)b1 << 16;
            }
            if (units >= 2 &&
                !(ok = wait_warp(&sm.q_empty[units & 1], ((units - 2) >> 1) & 1)))
                break;
            if (h < kHeads) {
                uint8_t* q = sm.q[units & 1];
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const int chunk = part * kChunks + c;
                    *reinterpret_cast<uint4*>(q + swz<D>(h, chunk)) =
                        make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
                    *reinterpret_cast<uint4*>(q + swz<D>(kHeads + h, chunk)) =
                        make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
                }
                if (part == 0) sm.q_pow[units % kQPow][h] = __int_as_float((127 - e) << 23);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm.q_full[units & 1]);
        }
        // the last arrivals on the two buffers' barriers come before the CTA ends
        for (uint32_t i = 1; ok && i <= 2 && i <= units; ++i)
            ok = wait_warp(&sm.q_empty[(units - i) & 1], ((units - i) >> 1) & 1);
        if (!ok && lane == 0) give_up();
    } else if constexpr (!kGather) {
        // -------------------------------------------------------- TMA producer
        if (lane == 0) {
            tc::tma_prefetch_desc(&kmap);
            tc::tma_prefetch_desc(&vmap);
        }
        Ring ring;
        int issued = 0, units = 0;
        bool ok = true;
        // Lane l has box l of the unit (at most 2048 keys: 32 boxes).  Lanes 2j and
        // 2j + 1 (four lanes for head_dim 64) fill stage j, so a stage costs no shuffles
        // or divisions.  A unit needs its record, then its boxes' block ids, then their
        // scales: at a unit's start the next one's scales, the ids of the one after and
        // the record of the third are requested, and have that unit's time to arrive.
        auto load_block = [&](const int4& i) {
            const int32_t kk = i.y + lane * kBoxKeys;
            return kk < i.z ? a.bt[(int64_t)i.x * a.MB + kk / a.bs] : -2;      // -2: past the end
        };
        auto load_scale = [&](const float* scales, int32_t blk, int32_t kvh) {
            return (unsigned)blk < (unsigned)a.NB ? __ldg(scales + (int64_t)blk * a.Hkv + kvh)
                                                  : 0.f;
        };
        const Schedule sched(a);
        Units un(a), next_un = un, third = un;
        int4 info = sched.record(un.sc);
        next_un.next();
        int4 next_info = sched.record(next_un.sc);
        third.next();
        third.next();
        int4 third_info = sched.record(third.sc);
        int32_t blk = load_block(info), next_blk = load_block(next_info);
        float ks_in = load_scale(fa.ks, blk, un.kv_head());
        float vs_in = load_scale(fa.vs, blk, un.kv_head());
        while (un.sc < sched.chunks && ok) {
            const int32_t kvh = un.kv_head();
            const int32_t key0 = info.y, keys = info.z - key0;
            const bool inside = (unsigned)blk < (unsigned)a.NB;
            const bool good = inside && pkv::scale_ok(ks_in) && pkv::scale_ok(vs_in);
            if (!good && blk != -2)
                pkv::report(a.status, inside ? PKV_STATUS_BAD_SCALE : PKV_STATUS_BAD_BLOCK_ID);
            const float ks = good ? ks_in : 0.f;
            const float lv = good ? __log2f(vs_in) : -INFINITY;
            // (good to 2^-22; __frsqrt_rn cost 1.5 us of 77 where every key has one)
            const float rv = good ? 0.25f * rsqrtf(vs_in) : 0.f;
            const uint32_t goods = __ballot_sync(0xffffffffu, good);
            const int32_t row = blk * a.bs + (key0 + lane * kBoxKeys) % a.bs;
            StageMeta m;
            const int32_t hg = un.head_group();
            m.h0 = kvh * a.G + hg * kMaxGroup;
            m.nh = min(kMaxGroup, a.G - hg * kMaxGroup);
            m.nch = info.w;
            m.row = (info.w == 1 ? info.x : un.sc) * a.Hq;
            m.n = (keys + kStageKeys - 1) / kStageKeys;
            m.unit = units++;
            // requests for the units after
            ks_in = load_scale(fa.ks, next_blk, next_un.kv_head());
            vs_in = load_scale(fa.vs, next_blk, next_un.kv_head());
            const int32_t third_blk = load_block(third_info);
            Units fourth = third;
            fourth.next();
            const int4 fourth_info = sched.record(fourth.sc);
            for (int j = 0; j * kStageKeys < keys; ++j) {
                if (!(ok = wait_warp(&sm.empty[ring.slot], ring.phase ^ 1))) break;
                const int i = lane - kBoxes * j; // 0 .. kBoxes - 1: its box is in the stage
                const bool in_stage = i >= 0 && i < kBoxes;
                if (in_stage) {
                    sm.ks[ring.slot][i] = ks;
                    sm.lv[ring.slot][i] = lv;
                    sm.rv[ring.slot][i] = rv;
                    if (i == 0) {
                        m.j = j;
                        m.keys = keys - j * kStageKeys;
                        sm.meta[ring.slot] = m;
                    }
                }
                __syncwarp();
                const uint32_t bytes = __popc(goods >> (kBoxes * j) & ((1u << kBoxes) - 1u)) *
                                       (2 * kBoxKeys * D);
                if (i == 0) {
                    if (bytes == 0)
                        tc::mbar_arrive(&sm.full[ring.slot]);
                    else
                        tc::mbar_expect_tx(&sm.full[ring.slot], bytes);
                }
                __syncwarp();
                if (in_stage && good) {
                    uint8_t* kt = sm.kv[ring.slot] + i * kBoxKeys * D;
                    tc::tma_load_3d(kt, &kmap, &sm.full[ring.slot], 0, kvh, row);
                    tc::tma_load_3d(kt + kTileBytes, &vmap, &sm.full[ring.slot], 0, kvh, row);
                }
                ++issued;
                ring.next();
            }
            un = next_un;
            info = next_info;
            blk = next_blk;
            next_un = third;
            next_info = third_info;
            next_blk = third_blk;
            third = fourth;
            third_info = fourth_info;
        }
        int ended = 0;                           // an end mark for either group
        for (; ok && ended < kGroups; ++ended) {
            Ring mark = ring;
            mark.next(ended);
            if (!(ok = wait_warp(&sm.empty[mark.slot], mark.phase ^ 1))) break;
            if (lane == 0) {
                sm.meta[mark.slot].n = 0;
                tc::mbar_arrive(&sm.full[mark.slot]);
            }
            __syncwarp();
        }
        if (!ok && lane == 0) give_up();
        // every copy issued has landed, and every slot's last release has arrived
        // (or, where a role gave up, never will), before the CTA ends.  A marked
        // slot was released before its mark, and its barrier has moved on.
        for (int i = 1; i <= min(issued, kStages - ended); ++i) {
            int s = ring.slot - i;
            uint32_t ph = ring.phase;
            if (s < 0) {
                s += kStages;
                ph ^= 1;
            }
            tc::mbar_drain(&sm.full[s], ph);
            if (ok && !(ok = wait_warp(&sm.empty[s], ph)) && lane == 0) give_up();
        }
    } else {
        // ------------------------------------------------- gathering producers
        // Team t takes stages t, t + kTeams, ...; a team's warp has half the rows of
        // each, lane l looks up rows l, l + 32, ... of them.  A team hands a stage over when
        // its copies have landed; meanwhile the other teams' are in flight.
        const int team = (warp - kFirstProducer) / kTeamWarps;
        const int row0 = (warp - kFirstProducer) % kTeamWarps * kGatherRows;
        constexpr int kRows = kGatherRows / 32;  // rows that a lane looks up
        Ring ring;
        int units = 0;
        bool ok = true;
        // A walk over the stages, with this lane's keys of each as table entry and
        // offset; a stage on is 128 keys on (divisions only at a unit's start).
        const int32_t step_blocks = kStageKeys / a.bs, step_off = kStageKeys % a.bs;
        const Schedule sched(a);
        Units un(a);
        int4 info = sched.record(un.sc), ahead;          // this unit's record and the next one's
        int32_t k = 0, block[kRows], off[kRows];
        auto start_unit = [&]() {
            Units after = un;
            after.next();
            ahead = sched.record(after.sc);
            k = info.y;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                block[i] = (k + row0 + lane + 32 * i) / a.bs;
                off[i] = (k + row0 + lane + 32 * i) % a.bs;
            }
        };
        auto step = [&]() {                      // to the CTA's next stage
            ring.next();
            k += kStageKeys;
            if (k >= info.z) {
                un.next();
                info = ahead;
                ++units;
                start_unit();
                return;
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                block[i] += step_blocks;
                off[i] += step_off;
                if (off[i] >= a.bs) {
                    off[i] -= a.bs;
                    ++block[i];
                }
            }
        };
        int32_t blk[kRows];                      // block ids; -2: past the end
        auto load_blocks = [&]() {
#pragma unroll
            for (int i = 0; i < kRows; ++i)
                blk[i] = k + row0 + lane + 32 * i < info.z
                             ? a.bt[(int64_t)info.x * a.MB + block[i]] : -2;
        };
        start_unit();
        for (int i = 0; i < team && un.sc < sched.chunks; ++i) step();
        load_blocks();
        while (un.sc < sched.chunks) {
            const int32_t kvh = un.kv_head();
            float ks[kRows], vs[kRows];
            // rows of one head: K and V within the GPU's memory have fewer than
            // 2^32 - 1 of them each
            uint32_t row[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                ks[i] = vs[i] = 0.f;
                row[i] = 0xffffffffu;
                if ((unsigned)blk[i] < (unsigned)a.NB) {
                    const int64_t at = (int64_t)blk[i] * a.Hkv + kvh;
                    ks[i] = __ldg(fa.ks + at);
                    vs[i] = __ldg(fa.vs + at);
                    row[i] = ((uint32_t)blk[i] * (uint32_t)a.bs + (uint32_t)off[i]) *
                                 (uint32_t)a.Hkv + (uint32_t)kvh;
                }
            }
            if (!(ok = wait_warp(&sm.empty[ring.slot], ring.phase ^ 1))) break;
            const int slot = ring.slot;
            uint8_t* kt = sm.kv[slot] + row0 * D;
            constexpr int kChunks = D / 16, kAtOnce = 32 / kChunks;      // of a row; rows a copy
#pragma unroll
            for (int j = 0; j < kGatherRows / kAtOnce; ++j) {
                const int r = kAtOnce * j + lane / kChunks, c = lane % kChunks;
                const uint32_t src = __shfl_sync(0xffffffffu, row[j * kAtOnce / 32], r & 31);
                const bool there = src != 0xffffffffu;
                const uint64_t at = there ? (uint64_t)src * D + c * 16 : 0;
                cp_async16(kt + swz<D>(r, c), fa.kc + at, there ? 16 : 0);
                cp_async16(kt + kTileBytes + swz<D>(r, c), fa.vc + at, there ? 16 : 0);
            }
            if (row0 == 0 && lane == 0) {
                StageMeta m;
                m.j = (k - info.y) / kStageKeys;
                m.n = (info.z - info.y + kStageKeys - 1) / kStageKeys;
                m.keys = info.z - k;
                m.unit = units;
                const int32_t hg = un.head_group();
                m.h0 = kvh * a.G + hg * kMaxGroup;
                m.nh = min(kMaxGroup, a.G - hg * kMaxGroup);
                m.nch = info.w;
                m.row = (info.w == 1 ? info.x : un.sc) * a.Hq;
                sm.meta[slot] = m;
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const bool inside = (unsigned)blk[i] < (unsigned)a.NB;
                const bool good = inside && pkv::scale_ok(ks[i]) && pkv::scale_ok(vs[i]);
                if (!good && blk[i] != -2)
                    pkv::report(a.status,
                                inside ? PKV_STATUS_BAD_SCALE : PKV_STATUS_BAD_BLOCK_ID);
                const int key = row0 + lane + 32 * i;
                sm.ks[slot][key] = good ? ks[i] : 0.f;
                sm.lv[slot][key] = good ? __log2f(vs[i]) : -INFINITY;
                sm.rv[slot][key] = good ? 0.25f * rsqrtf(vs[i]) : 0.f;
            }
            // the team's next stage: its block ids arrive while the copies land
            for (int i = 0; i < kTeams && un.sc < sched.chunks; ++i) step();
            load_blocks();
            asm volatile("cp.async.wait_all;" ::: "memory");
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm.full[slot]);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        // past the last stage: the ring stands behind it for every team.  The first
        // team marks the end for either group, and waits for the slots' last release.
        if (ok && team == 0) {
            for (int i = 0; ok && i < kGroups; ++i) {
                Ring mark = ring;
                mark.next(i);
                if (!(ok = wait_warp(&sm.empty[mark.slot], mark.phase ^ 1))) break;
                if (row0 == 0 && lane == 0) sm.meta[mark.slot].n = 0;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sm.full[mark.slot]);
            }
            for (int i = 1; ok && i <= kStages - kGroups; ++i) {
                const int s = ring.slot - i;
                const uint32_t phase = s < 0 ? ring.phase ^ 1 : ring.phase;
                if (s < 0 && ring.laps == 0) break;          // never filled
                ok = wait_warp(&sm.empty[s < 0 ? s + kStages : s], phase);
            }
        }
        if (!ok && lane == 0) give_up();
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kSWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

// Rows of [rows, heads, D] codes, one head of kBoxKeys rows a box.
template <int D>
bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int heads) {
    auto enc = pkv::tma_encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)heads * D};
    cuuint32_t box[3] = {(cuuint32_t)D, 1, (cuuint32_t)kBoxKeys};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
               es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int kHeads, bool kGather, bool kPolls>
int launch(const Fp8DecodeArgs& fa, cudaStream_t s) {
    const pkv::DecodeArgs& a = fa.d;
    CUtensorMap kmap{}, vmap{};
    const int64_t rows = (int64_t)a.NB * a.bs;
    if (!kGather && (!encode_rows<D>(&kmap, fa.kc, rows, a.Hkv) ||
                     !encode_rows<D>(&vmap, fa.vc, rows, a.Hkv)))
        return PKV_ERR_CUDA;
    const int smem = (int)sizeof(Smem<D>) + 1024;
    static std::atomic<uint64_t> configured{0};
    void (*kernel)(const CUtensorMap, const CUtensorMap, Fp8DecodeArgs) =
        decode_fp8_tc_kernel<D, kHeads, kGather, kPolls>;
    if (!pkv_dynamic_smem_once((const void*)kernel, smem, configured)) return PKV_ERR_CUDA;
    int64_t grid = pkv_num_sms();
    const int64_t upper = (int64_t)a.cap * a.Hkv * a.n_hg;
    if (grid > upper) grid = upper;
    if (grid < 1) grid = 1;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((kFirstProducer + (kGather ? kGatherWarps : 1)) * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, kmap, vmap, fa) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// Waits with a poll limit other than the default are an instantiation of their
// own; it takes any number of heads.
template <int D, bool kGather>
int launch_heads(const Fp8DecodeArgs& fa, cudaStream_t s) {
    if (fa.d.wait_polls != (uint32_t)PKV_DEFAULT_WAIT_POLLS)
        return launch<D, 8, kGather, true>(fa, s);
    if (fa.d.G <= 2) return launch<D, 2, kGather, false>(fa, s);
    if (fa.d.G <= 4) return launch<D, 4, kGather, false>(fa, s);
    return launch<D, 8, kGather, false>(fa, s);
}

template <int D>
int launch_blocks(const Fp8DecodeArgs& fa, cudaStream_t s) {
    const bool boxes = fa.d.bs % kBoxKeys == 0 && fa.d.chunk_keys % kBoxKeys == 0 &&
                       pkv::tma_encode_fn() != nullptr;
    return boxes ? launch_heads<D, false>(fa, s) : launch_heads<D, true>(fa, s);
}

}  // namespace

int pkv_launch_decode_fp8(const Fp8DecodeArgs& fa, int head_dim, cudaStream_t s) {
    return head_dim == 128 ? launch_blocks<128>(fa, s) : launch_blocks<64>(fa, s);
}
