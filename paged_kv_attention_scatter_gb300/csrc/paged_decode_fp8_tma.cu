// paged_decode_fp8 split kernel fed by TMA (block sizes that are multiples of
// 64).  The arithmetic is that of paged_decode_fp8.cu; the roles and bounded
// waits are those of the bf16 kernel in paged_decode_tma.cu:
//
//  * One CTA per SM, 9 warps.  Warp 8 is the producer: it walks the CTA's
//    units and fills a ring of 128-key stages (32 KB for head_dim 128), each as
//    two 64-key TMA boxes of K and two of V (a box lies in one cache block), plus
//    the unit's q rows on its first stage.  A box's two scales, fetched with
//    the block ids a unit ahead, ride in the stage's record.
//  * Warps 0-7 consume 16 keys each.  Half the bytes of a bf16 key arrive with
//    the same number of keys' worth of arithmetic plus the conversions, so the
//    consumers have about half the time a key that the bf16 kernel's have: eight
//    warps instead of four, on stages of twice the keys, hide each other's
//    latency.  A warp whose 16 keys are all past the end skips the arithmetic.
//  * Inside a warp's 16 keys, fragment key k sits at row k ^ ((k & 1) << 2):
//    with the 128-byte swizzle every 16-byte fragment load of K and of V is
//    free of bank conflicts (head_dim 64: 64-byte swizzle, the 8-byte V loads
//    are two-way).
//  * At a unit's end the warps' partial outputs cross shared memory in the order
//    their fragments have them (a padded row per head), which keeps those
//    stores free of conflicts; heads that the unit lacks are not written.
#include <cudaTypedefs.h>

#include "fp8_common.cuh"
#include "tc_utils.cuh"
#include "tma_host.cuh"

using pkv::Fp8DecodeArgs;
using pkv::kMaxGroup;

namespace {

namespace tc = pkv::tc;

constexpr int kBoxKeys = 64;
constexpr int kStageKeys = 2 * kBoxKeys;
constexpr int kConsumerWarps = kStageKeys / 16;
constexpr int kThreads = (kConsumerWarps + 1) * 32;

enum : int32_t { kFirst = 1, kLast = 2, kEnd = 4, kMasked0 = 8, kMasked1 = 16 };

struct StageMeta {
    int32_t b, flags, keys;              // keys: valid ones from the stage's first on
    int32_t sc, h0, nh, nch, pad;
    float ks[2], lv[2], iv[2];           // per box: K scale, log2 and inverse of V's
};

template <int D>
struct Cfg {
    static constexpr int kBoxBytes = kBoxKeys * D;
    static constexpr int kStageBytes = 4 * kBoxBytes;         // K boxes, then V boxes
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int kQBytes = kMaxGroup * D * 2;
    static constexpr int kRow = D + 4;                        // partial output row, padded
};

template <int D>
struct Smem {
    uint8_t kv[Cfg<D>::kStages][Cfg<D>::kStageBytes];         // 1024-byte aligned boxes
    uint8_t qs[Cfg<D>::kStages][Cfg<D>::kQBytes];
    StageMeta meta[Cfg<D>::kStages];
    uint64_t full[Cfg<D>::kStages];
    uint64_t empty[Cfg<D>::kStages];
    uint64_t merge_full;                                      // the warps' partials written
    uint64_t merge_free;                                      // ... and read by the merge
    float m[kConsumerWarps][kMaxGroup];
    float l[kConsumerWarps][kMaxGroup];
    float o[kConsumerWarps][kMaxGroup][Cfg<D>::kRow];
    int abort_flag;
};

__device__ __forceinline__ uint4 lds16(const uint8_t* p) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(tc::saddr(p)));
    return r;
}
__device__ __forceinline__ uint2 lds8(const uint8_t* p) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(tc::saddr(p)));
    return r;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(tc::saddr(dst)), "l"(src), "r"(bytes), "r"(tc::saddr(bar))
        : "memory");
}

// Row of fragment key k (0..15) inside a warp's 16.
__device__ __forceinline__ int key_row(int k) { return k ^ ((k & 1) << 2); }

// Byte offset of 16-byte chunk c of row r in a swizzled box of D-byte rows
// (128-byte swizzle: chunk ^ row; 64-byte: two rows a 128-byte line, chunk ^ line).
template <int D>
__device__ __forceinline__ int swz(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Position of head_dim entry d in a partial output row (fragment order: m-tile,
// then lane group, then the pair).
template <int D>
__device__ __forceinline__ int o_pos(int d) {
    constexpr int VE = D / 8;
    const int g = d / VE, e = d % VE;
    return (e >> 1) * 16 + 2 * g + (e & 1);
}

template <int D, bool kPolls>
__global__ void __launch_bounds__(kThreads, 1)
    decode_fp8_tma_kernel(const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, Fp8DecodeArgs fa) {
    const pkv::DecodeArgs& a = fa.d;
    const uint32_t polls = kPolls ? a.wait_polls : (uint32_t)PKV_DEFAULT_WAIT_POLLS;
    using C = Cfg<D>;
    constexpr int S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            tc::mbar_init(&sm.full[s], 1);
            tc::mbar_init(&sm.empty[s], kConsumerWarps);
        }
        tc::mbar_init(&sm.merge_full, kConsumerWarps * 32);
        tc::mbar_init(&sm.merge_free, kConsumerWarps * 32);
        sm.abort_flag = 0;
        tc::mbar_init_fence();
    }
    __syncthreads();
    pkv::wait_for_predecessor();                 // the plan kernel's chunk records
    pkv::allow_dependent_launch();

    const int units_per_sc = a.Hkv * a.n_hg;
    const int64_t units = (int64_t)a.chunk_prefix[a.B] * units_per_sc;
    // a bounded wait with one outcome for the whole warp
    auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, &sm.abort_flag, polls)) != 0;
    };

    if (warp == kConsumerWarps) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tc::tma_prefetch_desc(&kmap);
            tc::tma_prefetch_desc(&vmap);
        }
        int slot = 0;
        uint32_t phase = 0;
        int issued = 0;
        bool ok = true;
        // lane l holds the id and scales of the unit's l-th cache block (at most
        // 1024 keys: 17 blocks), loaded while the unit before is streamed
        auto head_of = [&](int64_t u) { return (int32_t)(u % units_per_sc) / a.n_hg; };
        auto load_block = [&](const int4& i) {
            const int32_t blk0 = i.y / a.bs, nblk = (i.z - 1) / a.bs - blk0 + 1;
            return lane < nblk ? a.bt[(int64_t)i.x * a.MB + blk0 + lane] : -1;
        };
        auto load_scale = [&](const float* scales, int32_t blk, int32_t kvh) {
            return (unsigned)blk < (unsigned)a.NB ? __ldg(scales + (int64_t)blk * a.Hkv + kvh)
                                                  : 0.f;
        };
        int64_t u = blockIdx.x;
        int4 info_next = make_int4(0, 0, 0, 0);
        int32_t blk_next = -1;
        float ks_next = 0.f, vs_next = 0.f;
        if (u < units) {
            info_next = a.chunk_info[u / units_per_sc];
            blk_next = load_block(info_next);
            ks_next = load_scale(fa.ks, blk_next, head_of(u));
            vs_next = load_scale(fa.vs, blk_next, head_of(u));
        }
        while (u < units && ok) {
            const int32_t sc = (int32_t)(u / units_per_sc);
            const int32_t rem = (int32_t)(u - (int64_t)sc * units_per_sc);
            const int32_t kvh = rem / a.n_hg, hg = rem - kvh * a.n_hg;
            const int4 info = info_next;
            const int32_t my_blk = blk_next;
            const float my_ks = ks_next, my_vs = vs_next;
            const bool my_scales = pkv::scale_ok(my_ks) && pkv::scale_ok(my_vs);
            const float my_lv = __log2f(my_vs), my_iv = __frcp_rn(my_vs);
            const int64_t un = u + gridDim.x;
            if (un < units) info_next = a.chunk_info[un / units_per_sc];
            const int32_t b = info.x, key0 = info.y, key_end = info.z, nch = info.w;
            const int32_t blk0 = key0 / a.bs;
            const int32_t h0 = kvh * a.G + hg * kMaxGroup;
            const int32_t nh = min(kMaxGroup, a.G - hg * kMaxGroup);
            for (int32_t k = key0; k < key_end; k += kStageKeys) {
                if (!wait_warp(&sm.empty[slot], phase ^ 1)) {
                    ok = false;
                    break;
                }
                int32_t blk[2], at[2];
                bool good[2], scales[2];
                float ks[2], lv[2], iv[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int32_t kj = min(k + j * kBoxKeys, key_end - 1);
                    const int32_t i = kj / a.bs;
                    at[j] = (k + j * kBoxKeys) - i * a.bs;
                    blk[j] = __shfl_sync(0xffffffffu, my_blk, i - blk0);
                    scales[j] = __shfl_sync(0xffffffffu, (int)my_scales, i - blk0);
                    ks[j] = __shfl_sync(0xffffffffu, my_ks, i - blk0);
                    lv[j] = __shfl_sync(0xffffffffu, my_lv, i - blk0);
                    iv[j] = __shfl_sync(0xffffffffu, my_iv, i - blk0);
                }
                if (lane == 0) {
                    const bool first = k == key0;
                    int32_t flags = (first ? kFirst : 0) |
                                    (k + kStageKeys >= key_end ? kLast : 0);
                    uint32_t bytes = first ? (uint32_t)(nh * D * 2) : 0u;
                    StageMeta& m = sm.meta[slot];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const bool there = k + j * kBoxKeys < key_end;
                        const bool inside = (unsigned)blk[j] < (unsigned)a.NB;
                        good[j] = there && inside && scales[j];
                        if (good[j]) {
                            bytes += 2 * C::kBoxBytes;
                        } else {
                            flags |= j ? kMasked1 : kMasked0;
                            if (there)
                                pkv::report(a.status, inside ? PKV_STATUS_BAD_SCALE
                                                             : PKV_STATUS_BAD_BLOCK_ID);
                        }
                        m.ks[j] = ks[j];
                        m.lv[j] = lv[j];
                        m.iv[j] = iv[j];
                    }
                    m.b = b;
                    m.flags = flags;
                    m.keys = key_end - k;
                    m.sc = sc;
                    m.h0 = h0;
                    m.nh = nh;
                    m.nch = nch;
                    if (bytes == 0) {
                        tc::mbar_arrive(&sm.full[slot]);
                    } else {
                        tc::mbar_expect_tx(&sm.full[slot], bytes);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (!good[j]) continue;
                            const int32_t row = blk[j] * a.bs + at[j];
                            tc::tma_load_3d(sm.kv[slot] + j * C::kBoxBytes, &kmap, &sm.full[slot],
                                            0, kvh, row);
                            tc::tma_load_3d(sm.kv[slot] + (2 + j) * C::kBoxBytes, &vmap,
                                            &sm.full[slot], 0, kvh, row);
                        }
                        if (first)
                            bulk_load(sm.qs[slot], a.q + ((int64_t)b * a.Hq + h0) * D,
                                      (uint32_t)(nh * D * 2), &sm.full[slot]);
                    }
                }
                __syncwarp();
                ++issued;
                if (++slot == S) {
                    slot = 0;
                    phase ^= 1;
                }
                if (un < units) {                // the next unit's blocks, then their scales
                    if (k == key0) blk_next = load_block(info_next);
                    if (k == key0 + kStageKeys || (k == key0 && k + kStageKeys >= key_end)) {
                        ks_next = load_scale(fa.ks, blk_next, head_of(un));
                        vs_next = load_scale(fa.vs, blk_next, head_of(un));
                    }
                }
            }
            u = un;
        }
        if (ok && wait_warp(&sm.empty[slot], phase ^ 1)) {
            if (lane == 0) {
                sm.meta[slot].flags = kEnd;
                tc::mbar_arrive(&sm.full[slot]);
            }
            __syncwarp();
        } else {
            if (lane == 0) {
                sm.abort_flag = 1;
                pkv::report(a.status, PKV_STATUS_WAIT_TIMEOUT);
            }
        }
        // wait until the consumers are done (they arrive at barrier 1 on every
        // way out); if any role gave up, let every copy still in flight land
        // before the CTA can exit
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
        if (sm.abort_flag) {
            for (int i = 1; i <= min(issued, S); ++i) {
                int s = slot - i;
                uint32_t ph = phase;
                if (s < 0) {
                    s += S;
                    ph ^= 1;
                }
                tc::mbar_drain(&sm.full[s], ph);
            }
        }
        return;
    }

    // ---------------------------------------------------------------- consumers
    constexpr int NC = D / 64;       // 16-byte chunks per lane of a K row
    constexpr int KK = D / 16;       // k-steps of S = Q K^T
    constexpr int MT = D / 16;       // m-tiles of O^T
    constexpr int VW = D / 32;       // code words per lane of a V row
    const int g = lane >> 2, t = lane & 3;
    const int box = warp / (kBoxKeys / 16);
    int k_row[2], v_row[4], v_key[4];
#pragma unroll
    for (int r = 0; r < 2; ++r) k_row[r] = 16 * warp + key_row(8 * r + g);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        v_key[r] = 16 * warp + key_row(2 * t + (r & 1) + 8 * (r >> 1));
        v_row[r] = v_key[r];
    }

    uint32_t qa[KK][2];
    float o[MT][4];
    float m_run = -INFINITY, l_run = 0.f, x_scale = 0.f;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) qa[kk][0] = qa[kk][1] = 0u;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;

    int slot = 0;
    uint32_t phase = 0;
    uint32_t merged = 0;                         // units merged so far
    while (true) {
        if (!wait_warp(&sm.full[slot], phase)) {
            if (lane == 0) {
                sm.abort_flag = 1;
                pkv::report(a.status, PKV_STATUS_WAIT_TIMEOUT);
            }
            break;
        }
        const StageMeta& st = sm.meta[slot];
        const int32_t flags = st.flags;
        if (flags & kEnd) break;
        if (flags & kFirst) {
            x_scale = a.scale_log2 *
                      pkv::load_q_f16<D>(reinterpret_cast<const __nv_bfloat16*>(sm.qs[slot]) +
                                             g * D, g < st.nh, t, qa);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
            m_run = -INFINITY;
            l_run = 0.f;
        }
        const int32_t b = st.b, sc = st.sc, h0 = st.h0, nh = st.nh, nch = st.nch;
        const int32_t lim = (flags & (box ? kMasked1 : kMasked0)) ? 0 : st.keys;
        if (16 * warp < lim) {                   // some key of this warp's counts
            const uint8_t* kt = sm.kv[slot];
            const uint8_t* vt = kt + 2 * C::kBoxBytes;
            const float kf = st.ks[box] * x_scale, lv = st.lv[box], iv = st.iv[box];
            // ---- fragments: K rows of fragment keys g, 8 + g; V rows 2t, 2t+1, 2t+8, 2t+9 ----
            uint4 kr[2][NC];
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < NC; ++i) kr[r][i] = lds16(kt + swz<D>(k_row[r], i * 4 + t));
            bool valid[4];
            uint32_t vr[4][VW];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                valid[r] = v_key[r] < lim;
#pragma unroll
                for (int c = 0; c < VW; ++c) vr[r][c] = 0u;
                if (valid[r]) {
                    if constexpr (D == 128) {
                        const uint4 w = lds16(vt + swz<D>(v_row[r], g));
                        vr[r][0] = w.x;
                        vr[r][1] = w.y;
                        vr[r][2] = w.z;
                        vr[r][3] = w.w;
                    } else {
                        const uint2 w = lds8(vt + swz<D>(v_row[r], g >> 1) + 8 * (g & 1));
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
                    pkv::e4m3x4_to_f16x4(pkv::word(kr[nt][kk >> 2], kk & 3), b0, b1);
                    pkv::mma_f16_16816(s[nt], qa[kk][0], 0u, qa[kk][1], 0u, b0, b1);
                }
            }
            // ---- online softmax (base 2) over fragment keys 2t, 2t+1, 8+2t, 9+2t ----
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                y[j] = valid[j] ? fmaf(s[j >> 1][j & 1], kf, lv) : -INFINITY;
            float mx = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            const float m_new = fmaxf(m_run, mx);
            const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
            const float alpha = (m_run == -INFINITY) ? 0.f : pkv::fast_exp2(m_run - m_use);
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = pkv::fast_exp2(y[j] - m_use);
            l_run = fmaf((p[0] + p[1]) + (p[2] + p[3]), iv, l_run * alpha);
            m_run = m_new;
            const float alpha_a = __shfl_sync(0xffffffffu, alpha, (2 * t) * 4);
            const float alpha_b = __shfl_sync(0xffffffffu, alpha, (2 * t + 1) * 4);
            const uint32_t b0 = pkv::pack_f16(p[0], p[1]);
            const uint32_t b1 = pkv::pack_f16(p[2], p[3]);
            // ---- O^T = V^T P^T ----
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
        // every register read from the slot has been consumed: release it
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.empty[slot]);
        if (++slot == S) {
            slot = 0;
            phase ^= 1;
        }
        if (!(flags & kLast)) continue;

        // ---- end of a unit: merge the warps (bounded mbarrier waits, so a warp
        // that gave up can never leave the others blocked) ----
        if (merged > 0 &&
            !wait_warp(&sm.merge_free, (merged - 1) & 1)) {
            sm.abort_flag = 1;
            pkv::report(a.status, PKV_STATUS_WAIT_TIMEOUT);
            break;
        }
        float lr = l_run;
        lr += __shfl_xor_sync(0xffffffffu, lr, 1);
        lr += __shfl_xor_sync(0xffffffffu, lr, 2);
        if (t == 0) {
            sm.m[warp][g] = m_run;
            sm.l[warp][g] = lr;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (2 * t + e >= nh) continue;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
                *reinterpret_cast<float2*>(&sm.o[warp][2 * t + e][mt * 16 + 2 * g]) =
                    make_float2(o[mt][e], o[mt][2 + e]);
        }
        tc::mbar_arrive(&sm.merge_full);
        if (!wait_warp(&sm.merge_full, merged & 1)) {
            sm.abort_flag = 1;
            pkv::report(a.status, PKV_STATUS_WAIT_TIMEOUT);
            break;
        }
        for (int idx = threadIdx.x; idx < nh * D; idx += kConsumerWarps * 32) {
            const int h = idx / D, d = idx - h * D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kConsumerWarps; ++w) M = fmaxf(M, sm.m[w][h]);
            float L = 0.f, O = 0.f;
            if (M != -INFINITY) {
#pragma unroll
                for (int w = 0; w < kConsumerWarps; ++w) {
                    const float mw = sm.m[w][h];
                    if (mw == -INFINITY) continue;
                    const float f = pkv::fast_exp2(mw - M);
                    L += sm.l[w][h] * f;
                    O += sm.o[w][h][o_pos<D>(d)] * f;
                }
            }
            const int64_t qh = (int64_t)b * a.Hq + h0 + h;
            if (nch == 1) {
                a.out[qh * D + d] = __float2bfloat16_rn(L > 0.f ? O / L : 0.f);
            } else {
                const int64_t pslot = (int64_t)sc * a.Hq + h0 + h;
                a.part_o[pslot * D + d] = O;
                if (d == 0) a.part_ml[pslot] = make_float2(M, L);
            }
        }
        tc::mbar_arrive(&sm.merge_free);
        ++merged;
    }
    // the consumers are done: let the producer check for copies in flight
    asm volatile("bar.arrive 1, %0;" ::"n"(kThreads) : "memory");
}

// Rows of [rows, heads, D] codes, one head of kBoxKeys rows a box.
bool encode_rows(CUtensorMap* m, const void* base, int64_t rows, int heads, int D) {
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

template <int D>
int launch(const Fp8DecodeArgs& fa, cudaStream_t s) {
    const pkv::DecodeArgs& a = fa.d;
    CUtensorMap kmap, vmap;
    const int64_t rows = (int64_t)a.NB * a.bs;
    if (!encode_rows(&kmap, fa.kc, rows, a.Hkv, D) || !encode_rows(&vmap, fa.vc, rows, a.Hkv, D))
        return PKV_ERR_CUDA;
    const int smem = (int)sizeof(Smem<D>) + 1024;
    static std::atomic<uint64_t> configured[2] = {0, 0};
    const bool custom = a.wait_polls != (uint32_t)PKV_DEFAULT_WAIT_POLLS;
    void (*kernel)(const CUtensorMap, const CUtensorMap, Fp8DecodeArgs) =
        custom ? decode_fp8_tma_kernel<D, true> : decode_fp8_tma_kernel<D, false>;
    if (!pkv_dynamic_smem_once((const void*)kernel, smem, configured[custom]))
        return PKV_ERR_CUDA;
    int64_t grid = pkv_num_sms();
    const int64_t upper = (int64_t)a.cap * a.Hkv * a.n_hg;
    if (grid > upper) grid = upper;
    if (grid < 1) grid = 1;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, kmap, vmap, fa) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

bool pkv_decode_fp8_tma_supported(const Fp8DecodeArgs& fa) {
    return fa.d.bs % kBoxKeys == 0 && fa.d.chunk_keys % kBoxKeys == 0 &&
           pkv::tma_encode_fn() != nullptr;
}

int pkv_launch_decode_fp8_tma(const Fp8DecodeArgs& fa, int head_dim, cudaStream_t s) {
    return head_dim == 128 ? launch<128>(fa, s) : launch<64>(fa, s);
}
