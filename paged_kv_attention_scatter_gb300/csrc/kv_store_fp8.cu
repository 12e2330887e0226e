// kv_store_fp8: quantise each new token's K and V rows to e4m3 and scatter
// them into a paged cache with one scale for each (cache block, kv head).
//
// For a block and head that the call stores rows into, with x the rows' entries:
//   c' = max(c, 2^e), e the least integer with max|x| <= 448 * 2^e, in [-64, 119];
//   a stored row's codes are e4m3(x / c'), nearest-even, saturating;
//   every other row of the block has its codes replaced by e4m3(code * c / c').
// c is the block's scale before the call; a row at offset 0 begins the block
// anew (a sequence fills its blocks in order), and then c counts as 0 and the
// other rows are left alone.  A power of two changes no significant bit of a
// code, so x / c' is exact before its one rounding, a row re-scaled because its
// block grew keeps its codes' bits except where they fall among the
// subnormals, and storing a sequence row by row gives the values that storing
// it at once does (up to those subnormals).  A scale with a full significand
// would gain at most one bit of range and round every earlier row again
// each time it grew.
//
// Design.  One CTA owns a (block, set of heads): it needs every row the call
// stores there before it can write the first code.  It takes each head's
// maximum while reading the rows once, into registers or shared memory, and
// writes codes from there; a block is shared by as many CTAs as let each keep
// all of its rows (a CTA with twice the rows it can keep takes three times as
// long, and is the launch's last).  A row's head segment is read as 16 bytes a lane (D/8 lanes) and
// written as 8.  Rows that are consecutive tokens in consecutive slots, as a
// sequence's always are, are addressed by their first; any others (duplicates:
// the last token of a slot is stored) through a list in shared memory.  How
// rows find their block, by the number of tokens:
//  * up to 2048: one launch, a CTA per token.  Each scans all slots (8 KB at
//    most, out of L2, in one round of loads) for its block's tokens; the CTAs of
//    the first of them share the block's heads, one CTA for a decode step's
//    few rows, up to 2 * Hkv for a block that a prefill chunk fills, and the
//    others leave.
//  * more: that scan is quadratic, so a first kernel links the runs of
//    consecutive tokens in each block into a list per block, and notes whether a
//    block's rows are one token after another in one slot after another, and the
//    last of them.  The store kernel's CTAs then know their rows after two round
//    trips, or walk the lists.  Blocks of few and of many rows are listed apart, so
//    that a call of many sequences with a token each has one CTA a block (43 us
//    for 4096; 305 with the CTAs of full blocks).
// Memory's part: 4 bytes read and 2 written per K/V entry pair.  16384 tokens of 16
// prompts (8 heads of 128, blocks of 256) take 25 us, 4.1 TB/s: three waves of CTAs,
// each waiting 1.5 us for its rows' place, 3-4 for the rows at the copy rate, and
// converting for 2; three CTAs an SM with their rows in shared memory against two
// with them in registers.
#include "fp8_common.cuh"

namespace {

constexpr int kThreads = 256;
// Row segments a lane keeps in registers: a decode step has one row a block, a
// prefill chunk 256 over 16 lane groups.
constexpr int kKeepScan = 4, kKeepList = 16;
constexpr int32_t kScanTokens = 2048;        // largest call of the scanning form

struct StoreArgs {
    const uint4* k;
    const uint4* v;
    uint8_t* kc;
    uint8_t* vc;
    float* ks;
    float* vs;
    const int32_t* slots;
    int32_t n, bs, Hkv, NB;
    int64_t num_slots;
    uint32_t* status;
    // list form: runs linked per block
    int32_t* count;                          // [2]: blocks of few rows, of many; minus 1
    int32_t* head;                           // [NB]: token that starts the block's last run, -1
    int8_t* in_line;                         // [NB]: 0 if a run has tokens not slot after slot
    int32_t* last;                           // [NB]: last token of a run (of the only one)
    int32_t* next;                           // [n]: start of the run linked before, -1
    int2* list;                              // [list_size]: blocks that get rows, a run of each;
    int32_t list_size;                       //  few rows from the front, many from the back
    int32_t few, most;                       // CTAs of a block of few rows; most of one of many
};

constexpr int kScanLoads = kScanTokens / kThreads;

__device__ __forceinline__ void cp_async16(uint4* to, const uint4* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits for all but the last `pending` groups.
__device__ __forceinline__ void cp_async_wait(int pending) {
    if (pending >= 3) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (pending == 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (pending == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The rows that a call stores into one block: `rows` of them, tokens
// token0 + i at offsets offset0 + i (dense), or as listed.
struct RowLists {
    int32_t winner[pkv::kFp8MaxBlockSize];   // offset -> last token stored there, -1
    int32_t token[pkv::kFp8MaxBlockSize];    // the rows, in no particular order
    int16_t offset[pkv::kFp8MaxBlockSize];
};
struct BlockRows {
    int32_t rows, token0, offset0;
    bool dense;
    uint32_t amax[kThreads / 8];             // per lane group
    float ratio[kThreads / 8];               // per pair in hand: old / new scale where it grew,
                                             // else -1 (the quotient may round to 0)
};

// Larger magnitudes of the bf16 pairs of a vector and of `m`, two 16-bit lanes.
__device__ __forceinline__ uint32_t amax8(uint32_t m, const uint4& w) {
    m = __vmaxu2(m, w.x & 0x7fff7fffu);
    m = __vmaxu2(m, w.y & 0x7fff7fffu);
    m = __vmaxu2(m, w.z & 0x7fff7fffu);
    return __vmaxu2(m, w.w & 0x7fff7fffu);
}

// The same of finite entries only.
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {
    const uint32_t lo = w & 0x7fffu, hi = w & 0x7fff0000u;
    return (lo < 0x7f80u ? lo : 0u) | (hi < 0x7f800000u ? hi : 0u);
}
__device__ __forceinline__ uint32_t finite_amax8(uint32_t m, const uint4& w) {
    return amax8(m, make_uint4(finite_pair(w.x), finite_pair(w.y), finite_pair(w.z),
                               finite_pair(w.w)));
}

// 2^e for the least e with (bf16 magnitude) <= 448 * 2^e, clamped.
__device__ __forceinline__ float scale_for(uint32_t mag) {
    const int e = (int)(mag >> 7) - 127 - ((mag & 0x7fu) <= 0x60u ? 8 : 7);  // 448 = 1.75 * 2^8
    const int c = min(max(e, pkv::kScaleExpLo), pkv::kScaleExpHi);
    return __int_as_float((c + 127) << 23);
}

// The codes of eight entries divided by the scale.  For a power of two that is
// a multiplication by its inverse; kDivide is for the scales of other writers.
template <bool kDivide>
__device__ __forceinline__ uint32_t two_codes(uint32_t w, float s) {
    const float lo = __int_as_float((int)(w << 16)), hi = __int_as_float((int)(w & 0xffff0000u));
    if constexpr (kDivide) return pkv::float2_to_e4m3x2(__fdiv_rn(lo, s), __fdiv_rn(hi, s));
    return pkv::float2_to_e4m3x2(lo * s, hi * s);
}
template <bool kDivide>
__device__ __forceinline__ uint2 eight_codes(const uint4& w, float s) {
    return make_uint2(two_codes<kDivide>(w.x, s) | two_codes<kDivide>(w.y, s) << 16,
                      two_codes<kDivide>(w.z, s) | two_codes<kDivide>(w.w, s) << 16);
}

__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float ratio) {
    uint32_t lo, hi;
    pkv::e4m3x4_to_f16x4(codes, lo, hi);
    const float2 a = pkv::f16x2_to_float2(lo), b = pkv::f16x2_to_float2(hi);
    return (uint32_t)pkv::float2_to_e4m3x2(a.x * ratio, a.y * ratio) |
           (uint32_t)pkv::float2_to_e4m3x2(b.x * ratio, b.y * ratio) << 16;
}

__device__ __forceinline__ void clear_rows(const StoreArgs& a, BlockRows& sm, RowLists& l) {
    for (int o = threadIdx.x; o < a.bs; o += kThreads) l.winner[o] = -1;
    if (threadIdx.x == 0) sm.rows = 0;
}

// The winners as a compact list (any order), between barriers.
__device__ __forceinline__ void list_rows(const StoreArgs& a, BlockRows& sm, RowLists& l) {
    __syncthreads();
    if (threadIdx.x == 0) sm.dense = false;
    for (int o = threadIdx.x; o < a.bs; o += kThreads) {
        const int32_t t = l.winner[o];
        if (t >= 0) {
            const int i = atomicAdd(&sm.rows, 1);
            l.token[i] = t;
            l.offset[i] = (int16_t)o;
        }
    }
    __syncthreads();
}

// Stores the rows of block `blk` for the (tensor, head) pairs part, part +
// parts, ... of the 2 * Hkv.  Pair p is head p >> 1 of K (even) or V.
// A lane's first kKeep row segments stay in registers, or in `staged` if that is given
// (a place of its own there, so no barrier).
template <int D, int kKeep, bool kDense, bool kStaged>
__device__ __forceinline__ void store_block(const StoreArgs& a, BlockRows& sm, const RowLists& l,
                                            uint4* staged, int32_t blk, int part, int parts) {
    constexpr int kLanes = D / 8;            // lanes of a row's head segment
    constexpr int kGroups = kThreads / kLanes;
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int pairs = 2 * a.Hkv;
    const int mine = (pairs - part + parts - 1) / parts;
    // groups per pair: a power of two, so a pair's groups are aligned
    int gpp = kGroups;
    while (gpp > 1 && kGroups / gpp < mine) gpp >>= 1;
    const int at_once = kGroups / gpp, sub = group % gpp;
    const int rows = sm.rows;
    const int32_t token0 = sm.token0, offset0 = sm.offset0;
    const bool fresh = kDense ? offset0 == 0 : l.winner[0] >= 0;
    const int64_t row_codes = (int64_t)a.Hkv * D;
    auto token_of = [&](int r) { return kDense ? token0 + r : l.token[r]; };
    auto offset_of = [&](int r) { return kDense ? offset0 + r : (int)l.offset[r]; };
    // rows of the block that this call does not store
    auto other = [&](int o) {
        return kDense ? o < offset0 || o >= offset0 + rows : l.winner[o] < 0;
    };
    for (int i0 = 0; i0 < mine; i0 += at_once) {
        const int i = i0 + group / gpp;
        const bool live = i < mine;
        const int pair = part + (live ? i : 0) * parts;
        const int h = pair >> 1;
        const uint4* src = ((pair & 1) ? a.v : a.k) + h * kLanes + lane;
        uint8_t* dst = ((pair & 1) ? a.vc : a.kc) + (int64_t)blk * a.bs * row_codes + h * D +
                       lane * 8;
        float* scale_at = ((pair & 1) ? a.vs : a.ks) + (int64_t)blk * a.Hkv + h;
        auto load = [&](int r) { return __ldg(src + (int64_t)token_of(r) * (row_codes / 8)); };
        // ---- the pair's maximum; the first kKeep rows stay in registers ----
        const int n = live ? rows : 0;
        uint4 keep[kStaged ? 1 : kKeep];
        uint4* const mine_at = staged + threadIdx.x;
        constexpr int kPart = kKeep / 4;     // rows waited for at once
        const uint4* from = src + (int64_t)(token0 + sub) * (row_codes / 8);   // dense rows
#pragma unroll
        for (int j = 0; j < kKeep; ++j) {
            const bool there = sub + j * gpp < n;
            if constexpr (kStaged) {
                if (there) cp_async16(mine_at + j * kThreads, from);
                if (j % kPart == kPart - 1) cp_async_commit();
            } else {
                keep[j] = make_uint4(0, 0, 0, 0);
                if (there) keep[j] = kDense ? __ldg(from) : load(sub + j * gpp);
            }
            from += gpp * (row_codes / 8);
        }
        float old = 0.f;
        if (live && !fresh) old = *scale_at;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kKeep; ++j) {
            if constexpr (kStaged) {
                if (j % kPart == 0) cp_async_wait(kKeep / kPart - 1 - j / kPart);
                if (sub + j * gpp < n) m = amax8(m, mine_at[j * kThreads]);
            } else {
                m = amax8(m, keep[j]);
            }
        }
        const int rest = sub + kKeep * gpp;
#pragma unroll 4
        for (int r = rest; r < n; r += gpp) m = amax8(m, load(r));
        if ((m & 0x7fffu) >= 0x7f80u || m >= 0x7f800000u) {      // infinities or NaN
            m = 0;
#pragma unroll 1
            for (int r = sub; r < n; r += gpp) m = finite_amax8(m, load(r));
        }
        m = max(m & 0xffffu, m >> 16);
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1)
            m = max(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (gpp > 1) {
            if (lane == 0) sm.amax[group] = m;
            __syncthreads();                 // every group has read its old scale too
            for (int g = 0; g < gpp; ++g) m = max(m, sm.amax[group - sub + g]);
        }
        float ratio = -1.f;
        if (live) {
            if (!(old == 0.f || pkv::scale_ok(old))) {
                if (lane == 0 && sub == 0) pkv::report(a.status, PKV_STATUS_BAD_SCALE);
                old = 0.f;
            }
            const float scale = fmaxf(old, scale_for(m));
            auto at = [&](int r) {
                return reinterpret_cast<uint2*>(dst + offset_of(r) * row_codes);
            };
            if ((__float_as_int(scale) & 0x7fffff) == 0) {
                const float inv = __fdiv_rn(1.f, scale);
                uint8_t* to = dst + (offset0 + sub) * row_codes;
#pragma unroll
                for (int j = 0; j < kKeep; ++j) {
                    if (sub + j * gpp < n)
                        *(kDense ? reinterpret_cast<uint2*>(to) : at(sub + j * gpp)) =
                            eight_codes<false>(
                                kStaged ? mine_at[j * kThreads] : keep[kStaged ? 0 : j], inv);
                    to += gpp * row_codes;
                }
#pragma unroll 4
                for (int r = rest; r < n; r += gpp) *at(r) = eight_codes<false>(load(r), inv);
            } else {
#pragma unroll 1
                for (int r = sub; r < n; r += gpp) *at(r) = eight_codes<true>(load(r), scale);
            }
            if (old > 0.f && scale > old) ratio = __fdiv_rn(old, scale);
            if (lane == 0 && sub == 0) *scale_at = scale;
        }
        if (lane == 0 && sub == 0) sm.ratio[group / gpp] = ratio;
        // (this barrier also lets the next round's maxima be written)
        if (!__syncthreads_or(ratio >= 0.f)) continue;
        // ---- blocks that grew: their other rows, the whole CTA on one pair at a
        // time (a decode step's pair has one lane group, and 256 rows one after
        // another would take as long as the rest of the step) ----
        for (int p = 0; p < at_once; ++p) {
            const float r = sm.ratio[p];
            if (!(r >= 0.f)) continue;
            const int pr = part + (i0 + p) * parts;
            uint8_t* base = ((pr & 1) ? a.vc : a.kc) + (int64_t)blk * a.bs * row_codes +
                            (pr >> 1) * D + lane * 8;
            constexpr int kBatch = 8;
            for (int o0 = group; o0 < a.bs; o0 += kBatch * kGroups) {
                uint2 c[kBatch];
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int o = o0 + j * kGroups;
                    if (o < a.bs && other(o))
                        c[j] = *reinterpret_cast<const uint2*>(base + o * row_codes);
                }
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int o = o0 + j * kGroups;
                    if (o < a.bs && other(o))
                        *reinterpret_cast<uint2*>(base + o * row_codes) =
                            make_uint2(rescale4(c[j].x, r), rescale4(c[j].y, r));
                }
            }
        }
        __syncthreads();                     // sm.ratio is read before the next round
    }
}

// CTAs that share a block's pairs: as many as let each keep all of its rows.
template <int D, int kKeep>
__host__ __device__ __forceinline__ int parts_of(int rows, int pairs) {
    constexpr int kGroups = kThreads / (D / 8);
    int gpp = 1;                             // lane groups a pair needs
    while (gpp < kGroups && gpp * kKeep < rows) gpp <<= 1;
    const int mine = kGroups / gpp;
    return (pairs + mine - 1) / mine;
}

// Up to kScanTokens tokens: CTA t belongs to token t.
template <int D>
__global__ void __launch_bounds__(kThreads, 4) store_scan_kernel(StoreArgs a) {
    __shared__ BlockRows sm;
    __shared__ RowLists lists;
    __shared__ int32_t before, total, first_token, first_slot;
    pkv::allow_dependent_launch();
    const int32_t t = blockIdx.x;
    int32_t s[kScanLoads];
#pragma unroll
    for (int j = 0; j < kScanLoads; ++j) {
        const int32_t i = threadIdx.x + j * kThreads;
        s[j] = i < a.n ? __ldg(a.slots + i) : -1;
    }
    const int32_t slot = a.slots[t];
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        if (threadIdx.x == 0) pkv::report(a.status, PKV_STATUS_SLOT_OUT_OF_RANGE);
        return;
    }
    const int32_t blk = slot / a.bs;
    const int32_t lo = blk * a.bs, hi = lo + a.bs;
    if (threadIdx.x == 0) {
        before = total = 0;
        first_token = INT_MAX;
    }
    __syncthreads();
    int b = 0, all = 0;
    int32_t first = INT_MAX;
#pragma unroll
    for (int j = kScanLoads - 1; j >= 0; --j) {
        if (s[j] < lo || s[j] >= hi) continue;
        const int32_t i = threadIdx.x + j * kThreads;
        first = i;
        ++all;
        b += i < t;
    }
    if (all) {
        atomicAdd(&total, all);
        atomicAdd(&before, b);
        atomicMin(&first_token, first);
    }
    __syncthreads();
    const int rows = total, part = before;
    const int parts = min(rows, parts_of<D, kKeepScan>(rows, 2 * a.Hkv));
    if (part >= parts) return;
    if (threadIdx.x == first_token % kThreads) first_slot = a.slots[first_token];
    __syncthreads();
    // dense: the block's tokens are first_token + i in slots first_slot + i
    bool in_line = true;
#pragma unroll
    for (int j = 0; j < kScanLoads; ++j) {
        const int32_t i = threadIdx.x + j * kThreads;
        if (s[j] >= lo && s[j] < hi)
            in_line = in_line && i - first_token == s[j] - first_slot && i - first_token < rows;
    }
    if (__syncthreads_and(in_line)) {
        if (threadIdx.x == 0) {
            sm.dense = true;
            sm.rows = rows;
            sm.token0 = first_token;
            sm.offset0 = first_slot - lo;
        }
        __syncthreads();
    } else {
        clear_rows(a, sm, lists);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kScanLoads; ++j)
            if (s[j] >= lo && s[j] < hi)
                atomicMax(&lists.winner[s[j] - lo], (int32_t)threadIdx.x + j * kThreads);
        list_rows(a, sm, lists);
    }
    if (sm.dense)
        store_block<D, kKeepScan, true, false>(a, sm, lists, nullptr, blk, part, parts);
    else
        store_block<D, kKeepScan, false, false>(a, sm, lists, nullptr, blk, part, parts);
}

// More tokens: each block's runs as a linked list, and the blocks as a list.
__global__ void __launch_bounds__(kThreads) store_link_kernel(StoreArgs a) {
    pkv::allow_dependent_launch();
    const int32_t t = blockIdx.x * kThreads + threadIdx.x;
    if (t >= a.n) return;
    const int32_t slot = a.slots[t];
    const int32_t prev = t > 0 ? a.slots[t - 1] : -1, next = t < a.n - 1 ? a.slots[t + 1] : -1;
    const int32_t ahead = t < a.n - kKeepList ? a.slots[t + kKeepList] : -1;
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        pkv::report(a.status, PKV_STATUS_SLOT_OUT_OF_RANGE);
        return;
    }
    const int32_t blk = slot / a.bs, lo = blk * a.bs, hi = lo + a.bs;
    if (next < lo || next >= hi) a.last[blk] = t;
    if (prev >= lo && prev < hi) {           // inside a run
        if (slot != prev + 1) a.in_line[blk] = 0;
        return;
    }
    const int32_t linked = atomicExch(&a.head[blk], t);
    a.next[t] = linked;
    if (linked >= 0) return;
    // more rows than a lane group keeps, if the run is in line
    const bool many = ahead >= 0 && ahead < hi && ahead - slot == kKeepList;
    const int32_t at = atomicAdd(a.count + many, 1) + 1;
    a.list[many ? a.list_size - 1 - at : at] = make_int2(blk, t);
}

constexpr int kListSmem = kKeepList * kThreads * 16;
constexpr int kListCtas = 3;
static_assert(kListSmem >= (int)sizeof(RowLists), "the lists take the staged rows' place");

// (out of line: its registers are not the dense rows' to give)
template <int D>
__device__ __noinline__ void store_listed(const StoreArgs& a, BlockRows& sm, const RowLists& l,
                                          int32_t blk, int part, int parts) {
    store_block<D, kKeepScan, false, false>(a, sm, l, nullptr, blk, part, parts);
}

template <int D>
__global__ void __launch_bounds__(kThreads, kListCtas) store_list_kernel(StoreArgs a) {
    extern __shared__ __align__(16) char dynamic[];          // staged rows, or the lists
    __shared__ BlockRows sm;
    uint4* const staged = reinterpret_cast<uint4*>(dynamic);
    RowLists& lists = *reinterpret_cast<RowLists*>(dynamic);
    pkv::wait_for_predecessor();             // the linked runs
    pkv::allow_dependent_launch();
    const uint32_t few = a.few, most = a.most;
    // (read beside the counts, and not used if there is no such entry)
    int2 entry = a.list[max(a.list_size - 1 - (int32_t)(blockIdx.x / most), 0)];
    // blocks * parts < 2^32, as the rows of n tokens fit a GPU's memory
    const uint32_t from_many = (uint32_t)(a.count[1] + 1) * most;
    const uint32_t items = from_many + (uint32_t)(a.count[0] + 1) * few;
    for (uint32_t i = blockIdx.x; i < items; i += gridDim.x) {
        const bool many = i < from_many;
        const uint32_t j = many ? i : i - from_many, of = many ? most : few;
        if (!many) entry = a.list[j / of];
        else if (i != blockIdx.x) entry = a.list[a.list_size - 1 - (int32_t)(j / of)];
        const int32_t blk = entry.x, run = entry.y;
        const int part = (int)(j % of);
        const int32_t lo = blk * a.bs, hi = lo + a.bs;
        const int32_t head = a.head[blk], slot0 = a.slots[run], last = a.last[blk];
        if (head == run && a.in_line[blk] != 0) {        // the block's only run
            if (threadIdx.x == 0) {
                sm.dense = true;
                sm.rows = last - run + 1;
                sm.token0 = run;
                sm.offset0 = slot0 - lo;
            }
            __syncthreads();
        } else {
            clear_rows(a, sm, lists);
            __syncthreads();
            for (int32_t r = head; r >= 0; r = a.next[r]) {
                // the run's tokens: up to the first one of another block
                for (int32_t j = r;; j += kThreads) {
                    const int32_t t = j + (int32_t)threadIdx.x;
                    const int32_t s = t < a.n ? a.slots[t] : -1;
                    const bool in = s >= lo && s < hi;
                    if (in) atomicMax(&lists.winner[s - lo], t);
                    if (!__syncthreads_and(in)) break;
                }
            }
            list_rows(a, sm, lists);
        }
        // a part beyond the rows' need has nothing to do
        const int parts = many ? parts_of<D, kKeepList>(sm.rows, 2 * a.Hkv) : (int)few;
        if (part < parts) {
            if (sm.dense)
                store_block<D, kKeepList, true, true>(a, sm, lists, staged, blk, part, parts);
            else
                store_listed<D>(a, sm, lists, blk, part, parts);
        }
        __syncthreads();                     // the rows in hand are read to the end
    }
}

struct StoreLayout {
    size_t off_head, off_in_line, off_last, off_next, off_list, total;
};

StoreLayout store_layout(int32_t n, int32_t num_blocks) {
    StoreLayout L{};
    if (n <= kScanTokens) return L;
    auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
    L.off_head = 16;                         // behind the counts, cleared with them
    L.off_in_line = L.off_head + sizeof(int32_t) * (size_t)num_blocks;   // cleared with them
    L.off_last = align(L.off_in_line + (size_t)num_blocks);
    L.off_next = align(L.off_last + sizeof(int32_t) * (size_t)num_blocks);
    L.off_list = align(L.off_next + sizeof(int32_t) * (size_t)n);
    L.total = align(L.off_list + sizeof(int2) * (size_t)(n < num_blocks ? n : num_blocks));
    return L;
}

template <int D>
int launch_store(const Fp8StoreCall& c, cudaStream_t s) {
    StoreArgs a{};
    a.k = (const uint4*)c.k;
    a.v = (const uint4*)c.v;
    a.kc = (uint8_t*)c.k_cache;
    a.vc = (uint8_t*)c.v_cache;
    a.ks = c.k_scale;
    a.vs = c.v_scale;
    a.slots = c.slot_mapping;
    a.n = c.num_tokens;
    a.bs = c.cache.block_size;
    a.Hkv = c.cache.num_kv_heads;
    a.NB = c.cache.num_blocks;
    a.num_slots = (int64_t)a.NB * a.bs;
    a.status = c.status;
    if (a.n <= kScanTokens) {
        store_scan_kernel<D><<<(unsigned)a.n, kThreads, 0, s>>>(a);
        return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
    }
    const StoreLayout L = store_layout(a.n, a.NB);
    char* ws = (char*)c.workspace;
    a.count = (int32_t*)ws;
    a.head = (int32_t*)(ws + L.off_head);
    a.in_line = (int8_t*)(ws + L.off_in_line);
    a.last = (int32_t*)(ws + L.off_last);
    a.next = (int32_t*)(ws + L.off_next);
    a.list = (int2*)(ws + L.off_list);
    a.list_size = a.n < a.NB ? a.n : a.NB;
    a.few = parts_of<D, kKeepList>(1, 2 * a.Hkv);
    a.most = parts_of<D, kKeepList>(a.bs, 2 * a.Hkv);
    if (cudaMemsetAsync(ws, 0xff, L.off_in_line + (size_t)a.NB, s) != cudaSuccess)
        return PKV_ERR_CUDA;
    store_link_kernel<<<(unsigned)((a.n + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
    static std::atomic<uint64_t> configured;
    if (!pkv_dynamic_smem_once((const void*)store_list_kernel<D>, kListSmem, configured))
        return PKV_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // about a CTA an item (blocks filled to half on average, at least): the
    // scheduler evens them out better than a loop does, and a CTA without one
    // leaves at once
    int64_t grid = 2LL * (a.n / a.bs + 1) * a.most;
    if (grid < pkv_num_sms() * 8) grid = pkv_num_sms() * 8;
    if (grid > 1 << 20) grid = 1 << 20;
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kListSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, store_list_kernel<D>, a) != cudaSuccess) return PKV_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

int pkv_kv_store_fp8_check(const Fp8StoreCall& c) {
    const pkv_cache_desc& d = c.cache;
    if (c.num_tokens < 0 || d.num_blocks <= 0 || d.block_size <= 0 || d.num_kv_heads <= 0)
        return PKV_ERR_BAD_DIMENSION;
    if (d.block_size > pkv::kFp8MaxBlockSize) return PKV_ERR_BAD_DIMENSION;
    if (d.head_dim != 64 && d.head_dim != 128) return PKV_ERR_UNSUPPORTED_HEAD_DIM;
    if ((int64_t)d.num_blocks * d.block_size >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;
    if (c.num_tokens == 0) return PKV_OK;
    if (!c.k || !c.v || !c.k_cache || !c.v_cache || !c.k_scale || !c.v_scale || !c.slot_mapping)
        return PKV_ERR_NULL_POINTER;
    if (((uintptr_t)c.k | (uintptr_t)c.v | (uintptr_t)c.k_cache | (uintptr_t)c.v_cache) & 15)
        return PKV_ERR_MISALIGNED;
    if (((uintptr_t)c.k_scale | (uintptr_t)c.v_scale | (uintptr_t)c.slot_mapping) & 3)
        return PKV_ERR_MISALIGNED;
    const size_t need = store_layout(c.num_tokens, d.num_blocks).total;
    if (need > 0) {
        if (!c.workspace) return PKV_ERR_NULL_POINTER;
        if ((uintptr_t)c.workspace & 15) return PKV_ERR_MISALIGNED;
        if (c.workspace_bytes < need) return PKV_ERR_WORKSPACE_TOO_SMALL;
    }
    return PKV_OK;
}

int pkv_kv_store_fp8_launch(const Fp8StoreCall& c, cudaStream_t s) {
    if (c.num_tokens == 0) return PKV_OK;
    return c.cache.head_dim == 128 ? launch_store<128>(c, s) : launch_store<64>(c, s);
}

extern "C" size_t pkv_kv_store_fp8_workspace_bytes(int32_t num_tokens, pkv_cache_desc cache) {
    if (num_tokens < 0 || cache.num_blocks <= 0) return 0;
    return store_layout(num_tokens, cache.num_blocks).total;
}

extern "C" int pkv_kv_store_fp8(const void* k, const void* v, void* k_cache, void* v_cache,
                                float* k_scale, float* v_scale, const int32_t* slot_mapping,
                                int32_t num_tokens, void* workspace, size_t workspace_bytes,
                                pkv_cache_desc cache, uint32_t* status, void* stream) {
    const Fp8StoreCall c{k, v, k_cache, v_cache, k_scale, v_scale, slot_mapping, num_tokens,
                         workspace, workspace_bytes, cache, status};
    const int rc = pkv_kv_store_fp8_check(c);
    return rc != PKV_OK ? rc : pkv_kv_store_fp8_launch(c, (cudaStream_t)stream);
}
