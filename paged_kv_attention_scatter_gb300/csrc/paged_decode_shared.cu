// paged_decode_shared: decode attention for a batch whose sequences come in groups with
// their first keys in common (one system prompt, one document, several samples of one
// prompt), the common keys read and multiplied once for up to 128 rows of a group's
// sequences, not once for each.
//
// What it computes: what paged_decode does,
//   out[b,h] = sum_{j < ctx_b} softmax_j(scale * q[b,h] . K_j) V_j.
// For a group of n sequences with P common keys the queries of one kv head are the
// n G rows of a matrix, so that Q K^T and P V over the common keys are matrix products
// of n G rows on the tensor cores.  A tile of 128 rows loads the common K and V rows; the further
// tiles of a larger group find most of them in L2 (256 sequences of four rows a head behind
// 8192 keys: eight tiles a head, 877 MB from DRAM in all where 824 cannot be avoided).  The
// softmax over a sequence's keys is put together from parts: each part is a maximum m, a sum l
// and an unnormalised o over some of the keys, and
//   M = max m,  out = sum 2^(m - M) o / sum 2^(m - M) l.
//
// Work item = (record, kv head, tile of q heads).  A record is a run of keys for up to 128
// rows: either common keys of some of a group's sequences, or own keys of one sequence.  Both
// go through the same kernel, so that items bound by the tensor cores (many rows on the same
// keys) and items bound by HBM (a few rows on keys of their own) run side by side.  One CTA
// of plan_kernel sizes the records from the lengths and lays them out; CTAs of the
// persistent attention kernel, one an SM, draw items from a counter.
//
// A CTA attends a 128-row tile against 128-key tiles, with the roles of the prefill's
// kernel (prefill_tc.cu, where the figures behind them stand):
//   warps 0-3  softmax: thread i owns row i = TMEM lane i.  P = exp2(S scale - m) is
//              computed against the running maximum straight away and goes over S in TMEM
//              as bf16, unnormalised: its rounding of 2^-8 of itself is that of a bf16
//              softmax, l is summed from the unrounded values.  Only for an item's first
//              tile, and where a row's sum passes 2^16 times its first weight, the maximum
//              is taken, O and l are rescaled and P computed again.
//   warp 4     producer: draws items, loads Q and K tiles (TMA, one box a run of a cache
//              block, or rows gathered with cp.async where the block size is no multiple
//              of 8) into a ring of three
//   warp 7     producer of the V tiles, likewise
//   warp 5, 6  issue Q K^T into one of three S buffers, and P V (tcgen05.mma)
// TMEM columns: S0 [0,128), S1 [128,256), S2 [256,384), O [384,384+D).
//
// What bounds it.  Own keys: the floor is their K and V rows once, but an item is a chain of
// waits (Q, first K tile, S, softmax, P V, epilogue) of about 2.5 us behind its tiles, and a
// tile costs one softmax warp about 1500 cycles, whatever few rows it has; with three items'
// worth of buffers in flight 256 sequences of 1..1500 keys run at 6.1 TB/s (129 us), 64 of 4096
// at 6.5.  Common keys: the softmax warps' pass over 128 x 128 scores, as in the prefill:
// 1260 TFLOP/s for 1024 sequences on 8192 keys, 1200 for 32 of 64 heads on 65536, 928 for 48 on
// two documents of 30000 and 65536, where a last wave of items and the parts show.  Both
// sorts together, 256 sequences with 8192 keys in common and up to 1500 of their own: 150 us,
// where the bytes take 123 and paged_decode 1160.  The softmax threads hold 255 registers (and
// spill 8 to 12 bytes), so an SM has one CTA and four softmax warps.  Forms that shorten an
// item by more instructions lost: own rows in quarters, one warp after another, 7 % (2 % gained
// for long ones), S^T with the keys in lanes 22 %, block ids asked for a tile ahead 3 to 9 %.
// What they share is 64 KB of code and more, of which a tile's part no longer stays in the
// nearest instruction cache (about 55 KB here); producers of fewer instructions gained 4 to
// 10 % everywhere.  head_dim 64 has the same scores to pass for half the bytes: 3.7 TB/s for 256
// sequences of 1..1500 keys.  Gathered rows (block sizes that are no multiple of 8) come at the
// pace of one warp's address arithmetic and copies: 2.6 TB/s there; blocks of 8 at 4.6.
//
// Keys outside a tile's run and keys of a block id outside the pool have weight 0, and
// their V rows are zeroed in shared memory, because unused cache slots may hold NaN.
// Every wait is bounded, as in the other tensor-core kernels: a wait that gives up sets
// PKV_STATUS_WAIT_TIMEOUT and the CTA unwinds once every copy and product it issued is done.
#include <cudaTypedefs.h>
#include <math.h>

#include "decode_common.cuh"
#include "tc_utils.cuh"
#include "tma_host.cuh"

using namespace pkv::tc;

namespace {

constexpr int kRows = 128;               // rows of a tile (TMEM lanes)
constexpr int kKeys = 128;               // key rows of a tile in shared memory
constexpr int kHalf = kKeys * 128;       // bytes of a tile's 64-column block
constexpr int kThreads = 256;
constexpr int kStages = 3;               // K, V and S buffers
constexpr int kItemRing = 4, kItemReaders = 7;
constexpr int kMaskRing = 8;             // more tiles than are between producer and softmax
constexpr uint32_t kColO = 384;
// P stands 2^-16 below 1 where a maximum is taken, and a maximum may be passed by 2^8 (a tile's
// sum by 2^16) before the next is: P and a tile's sum are 1 at most, so that P V passes V
// no further than the sum of a softmax's weights would.
constexpr float kHeadroom = 16.0f;
constexpr float kRescaleThreshold = 8.0f;
constexpr float kSumTrigger = 1.0f;
constexpr int kSms = 152;                // of a GB300: sizes follow from the arguments alone
constexpr int kMaxContext = 1 << 30;     // keys beyond it would pass 32 bits at a tile's end

// A run of keys for `seqs` sequences from b0 on, read through the table of sequence `table`
// (own keys: one sequence, and its table).
struct Record {
    int32_t b0, seqs, table, key_lo, key_hi;
    int32_t part;                        // place of its part among a sequence's
    int32_t origin, tiles;               // its tiles' first key; how many there are
};

// Division of 0 <= x < 2^31 by a d that the host knows: x m >> s with m = ceil(2^s / d) and
// s = 31 + ceil(log2 d), where m d - 2^s < d <= 2^(s - 31) makes the quotient exact.
struct Divisor {
    uint32_t m;
    int32_t s;
    __device__ __forceinline__ int32_t of(int32_t x) const {
        return (int32_t)(((uint64_t)(uint32_t)x * m) >> s);
    }
};

struct SharedArgs {
    const __nv_bfloat16* q;
    const __nv_bfloat16* kc;
    const __nv_bfloat16* vc;
    const int32_t* bt;
    __nv_bfloat16* out;
    int32_t* ctrl;                       // [0] records, [1] items drawn
    int32_t* part_prefix;                // [B + 1]: parts of the sequences before
    int2* sequences;                     // [B]: the plan's notes (see Sequence)
    int32_t* table;                      // [B], at a group's first sequence: whose table
    Record* records;
    float2* part_ml;                     // [cap_parts, Hq]: (max halved, sum)
    float* part_o;                       // [cap_parts, Hq, D]
    int32_t B, Hq, Hkv, G, MB, NB, bs, max_ctx, D;
    int32_t box, edge_box, tile_keys;    // rows of a TMA box; in tiles not full; keys of a tile
    int32_t tile_blocks, tile_rest;      // tile_keys in cache blocks, and keys beyond
    int32_t tile_heads, head_tiles, tile_seqs;
    int32_t cap_records, cap_parts, common_budget;
    float scale_log2;
    float far_unit, far_ratio;           // the power of two at or below it, their ratio (kFarScore)
    uint32_t* status;
    uint32_t wait_polls;
    // the plan's
    const int32_t* ctx;
    const int32_t* offsets;
    const int32_t* prefix;
    int32_t groups;
    Divisor by_box, by_tile, by_seqs;    // box, tile_keys, tile_seqs
};

__host__ __device__ __forceinline__ int32_t ceil_div(int32_t a, int32_t b) {
    return (a + b - 1) / b;
}

// ---------------------------------------------------------------------- plan
constexpr int kMaxPlanThreads = 1024;
constexpr int kStaged = 1024;            // groups held in shared memory
constexpr int kFew = 4;                  // groups up to which a length's items are counted exactly
// Fewer common keys than this are attended by each sequence itself.  64 sequences in 1, 8 and 32
// groups, up to 600 own keys, blocks of 16: 16 and 48 common keys together take 1 to 14 % longer
// than so; 80 to 240 between 13 % more (32 groups, 80 keys: 31.5 us for 28.1) and 8 % less (one
// group, 240: 29.9 for 32.5).  Without own keys any number is better together (9 us for 20), but
// a step's token itself is one.
constexpr int kMinShared = 64;
// What the plan expects, in ns: a key tile of common keys and of own ones (which come from
// HBM), the start and end of an item; and the bytes a ns of parts written and read again.  Taken
// from runs of one kind of item alone.  Any of them halved or doubled (the tiles' by 1.4),
// and the three quarters below as a half or as all, changes eight batches of all kinds by -4
// to +5 %, but for 256 sequences behind 8192 keys, where a common tile of 600, an own one of
// 2000, an item of 5000 and the half each choose longer common runs: 163 us for 151.
constexpr float kCommonTile = 850, kOwnTile = 1450, kItemCost = 2500, kPartBytes = 3500;

struct Group {
    int32_t first, seqs;
    int32_t prefix;                      // keys in common
    int32_t keys;                        // those attended together: all of them, or 0
};

// What a sequence attends: keys [0, prefix) with its group, [prefix, ctx) on its own.
struct Sequence {
    int32_t ctx, prefix;                 // ctx 0: nothing
};

// Groups as the plan reads them, the first kStaged from shared memory.
struct Groups {
    const SharedArgs& a;
    const int32_t* offsets;
    const int32_t* prefix;
    __device__ __forceinline__ Group at(int32_t g, bool report) const {
        Group x{offsets[g], 0, prefix[g], 0};
        x.seqs = offsets[g + 1] - x.first;
        if (x.prefix < 0 || x.prefix > (int64_t)a.MB * a.bs || x.prefix > a.max_ctx) {
            if (report) pkv::report(a.status, PKV_STATUS_BAD_SEQLENS);
            x.prefix = 0;
        }
        if (x.seqs >= 2 && x.prefix >= kMinShared) x.keys = x.prefix;
        return x;
    }
    // the group of sequence b among the first n, -1: none
    __device__ __forceinline__ int32_t of(int32_t b, int32_t n) const {
        int32_t lo = 0, hi = n;              // groups that begin at b or before
#pragma unroll 1
        while (lo < hi) {
            const int32_t mid = (lo + hi) / 2;
            if (offsets[mid] <= b) lo = mid + 1;
            else hi = mid;
        }
        return lo > 0 && b < offsets[lo] ? lo - 1 : -1;
    }
};

// The first key tile of a run begins at a box of the cache block that key_lo lies in.
__device__ __forceinline__ int32_t tile_origin(const SharedArgs& a, int32_t key_lo) {
    return a.by_box.of(key_lo) * a.box;
}
__device__ __forceinline__ int32_t key_tiles(const SharedArgs& a, int32_t lo, int32_t hi) {
    return hi > lo ? a.by_tile.of(hi - tile_origin(a, lo) + a.tile_keys - 1) : 0;
}
__device__ __forceinline__ int32_t row_tiles(const SharedArgs& a, int32_t seqs) {
    return a.by_seqs.of(seqs + a.tile_seqs - 1);
}

// Division of tile counts, 0 <= x <= 2^24, by a run length d <= 2^24: x + d - 1 and 1 / d are
// off by 2^-24 of themselves at most, the quotient by one then.
struct RunLength {
    int32_t d;
    float r;
    __device__ __forceinline__ explicit RunLength(int32_t n) : d(n), r(1.f / n) {}
    __device__ __forceinline__ int32_t runs(int32_t x) const {
        const int32_t y = x + d - 1;
        const int32_t q = __float2int_rz(__int2float_rn(y) * r), rest = y - q * d;
        return q + (rest >= d) - (rest < 0);
    }
};

// Block-wide exclusive prefix of v, over `carry` (updated to the sum).
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t& carry, int64_t* scratch) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[w] = x;
    __syncthreads();
    int64_t s = lane < (int)(blockDim.x >> 5) ? scratch[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, s, off);
        if (lane >= off) s += y;
    }
    const int64_t up = __shfl_sync(~0u, s, w > 0 ? w - 1 : 0);
    const int64_t all = __shfl_sync(~0u, s, 31);
    const int64_t r = carry + (w > 0 ? up : 0) + x - v;
    carry += all;
    return r;
}

// One CTA of a thread a sequence, within 256 and kMaxPlanThreads (for small batches more threads
// cost time: 64 sequences 6.4 us with 256, 8.2 with 1024, in an earlier form).  What a thread finds
// out of its first sequence stays in registers; larger batches go over theirs again.  Loops are
// not unrolled, divisions few and by products: a kernel that runs once pays for fetching its
// instructions (86 KB of them 16 us, 54 KB 7.0, 39 KB 5.5; two sequences as many as 64).
__global__ void __launch_bounds__(kMaxPlanThreads) plan_kernel(SharedArgs a) {
    pkv::allow_dependent_launch();
    __shared__ int64_t scratch[32];
    // common tiles of row tiles, of sequences; own tiles; row tiles; sequences with own keys
    __shared__ unsigned long long sum[5];
    __shared__ int32_t run_len[2];           // key tiles of a common run, of an own run
    __shared__ int32_t longest;              // key tiles of the longest prefix
    __shared__ int2 few[kFew];               // (row tiles, key tiles) of the first groups
    __shared__ int32_t staged_offsets[kStaged + 1], staged_prefix[kStaged], staged_table[kStaged];
    const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
    const int32_t units = a.Hkv * a.head_tiles;
    const int32_t my_ctx = tid < a.B ? a.ctx[tid] : 0;

    // ---- groups: increasing offsets within the batch, or none is used
    const bool staged = a.groups <= kStaged;
    if (tid < 5) sum[tid] = 0;
    if (tid == 5) longest = 1;
    if (staged && a.groups > 0)
#pragma unroll 1
        for (int32_t g = tid; g <= a.groups; g += threads) {
            staged_offsets[g] = a.offsets[g];
            if (g < a.groups) {
                staged_prefix[g] = a.prefix[g];
                staged_table[g] = INT32_MAX;
            }
        }
    __syncthreads();
    const Groups of{a, staged ? staged_offsets : a.offsets, staged ? staged_prefix : a.prefix};
    int32_t* table = staged ? staged_table : a.table;      // by group, or its first sequence
    bool bad = false;
    if (a.groups > 0)
#pragma unroll 1
        for (int32_t g = tid; g <= a.groups; g += threads) {
            const int32_t o = of.offsets[g];
            bad |= o < 0 || o > a.B || (g > 0 && o < of.offsets[g - 1]);
        }
    const int32_t groups = __syncthreads_or(bad) ? 0 : a.groups;
    if (groups != a.groups && tid == 0) pkv::report(a.status, PKV_STATUS_BAD_SEQLENS);

    // this thread's group of a round: neighbours go to different warps
    const int my_group = lane * (threads / 32) + (tid >> 5);
    // ---- how much there is
    auto add = [&](int which, int32_t v) {   // a warp's values into sum[which]
        v = __reduce_add_sync(~0u, v);
        if (lane == 0 && v != 0) atomicAdd(&sum[which], (unsigned long long)v);
    };
#pragma unroll 1
    for (int32_t base = 0; base < groups; base += threads) {
        const int32_t g = base + my_group;
        Group x{};
        if (g < groups) x = of.at(g, true);
        int32_t tiles = 0;
        int64_t t0 = 0, t1 = 0;              // these may pass 32 bits when added up
        int32_t n = 0;
        if (x.keys > 0) {
            tiles = row_tiles(a, x.seqs);
            n = key_tiles(a, 0, x.keys);
            atomicMax(&longest, n);
            if (!staged) a.table[x.first] = INT32_MAX;
            t0 = (int64_t)tiles * n;
            t1 = (int64_t)x.seqs * n;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            t0 += __shfl_xor_sync(~0u, t0, off);
            t1 += __shfl_xor_sync(~0u, t1, off);
        }
        if (lane == 0 && t0 != 0) {
            atomicAdd(&sum[0], (unsigned long long)t0);
            atomicAdd(&sum[1], (unsigned long long)t1);
        }
        if (g < kFew) few[g] = make_int2(tiles, n);
        add(3, tiles);
    }
    if (!staged) __syncthreads();
    Sequence mine{};                         // of sequence tid; the others' are noted
#pragma unroll 1
    for (int32_t base = 0; base < a.B; base += threads) {
        const int32_t b = base + tid;
        Sequence s{0, 0};
        if (b < a.B) {
            const int32_t c = base == 0 ? my_ctx : a.ctx[b];
            bool use = c > 0;
            if (c < 0 || c > (int64_t)a.MB * a.bs || c > a.max_ctx) {
                pkv::report(a.status, PKV_STATUS_BAD_CONTEXT_LEN);
                use = false;
            }
            const int32_t g = use ? of.of(b, groups) : -1;
            if (g >= 0) {
                const Group x = of.at(g, false);
                if (x.prefix > c) {          // a member without all of its group's keys
                    pkv::report(a.status, PKV_STATUS_BAD_CONTEXT_LEN);
                    use = false;
                } else if (x.keys > 0) {
                    s.prefix = x.keys;
                    atomicMin(&table[staged ? g : x.first], b);
                }
            }
            if (use) s.ctx = c;
        }
        if (base == 0) mine = s;
        else if (b < a.B) a.sequences[b] = make_int2(s.ctx, s.prefix);
        const int32_t own = key_tiles(a, s.prefix, s.ctx);
        add(2, own);
        add(4, own > 0);
    }
    auto noted = [&](int32_t b) {
        Sequence s = mine;
        if (b >= a.B) s = Sequence{};
        else if (b >= threads) {
            const int2 n = a.sequences[b];
            s = Sequence{n.x, n.y};
        }
        return s;
    };
    __syncthreads();

    // ---- run lengths
    if (tid < 32) {
        // (rounded up a little, so that 32 bits never give a run less than its share)
        const float common_tiles = (float)sum[0], members = (float)sum[1];
        const float own_tiles = (float)sum[2], work = own_tiles * units * (1 + 0x1p-20f);
        // own runs: an item's start and end cost as much as three tiles, so two items an SM up
        // to ten tiles each, then up to sixteen items (and no run longer than there can be)
        const float own_share = fmaxf(fminf(ceilf(work * (1.f / (2 * kSms))), 10.f),
                                      ceilf(work * (1.f / (16 * kSms))));
        const int32_t own = (int32_t)fminf(fmaxf(own_share, 1.f), kMaxContext / 64);
        const float own_cost = (own_tiles * kOwnTile +
                                (__fdividef(own_tiles, (float)own) + (float)sum[4]) * kItemCost) *
                               units;
        // a lane weighs two lengths: the longest prefix in so many runs, or in 1, 2, 3, ... tiles
        float best = INFINITY;
        int32_t chosen = 1;
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const int32_t len =
                k == 0 ? max(1, (int32_t)__fdividef((float)(longest + lane), lane + 1.f))
                       : lane < 8 ? lane + 1 : 2 * lane - 6;
            const float rcp = __fdividef(1.f, (float)len);
            float items = common_tiles * rcp + 0.5f * (float)sum[3];
            if (groups <= kFew) {
                int32_t count = 0;
#pragma unroll 1
                for (int32_t g = 0; g < groups; ++g)
                    count += few[g].x * (int32_t)((float)(few[g].y + len - 1) * rcp + 1e-3f);
                items = (float)count;
            }
            items *= units;
            const float item = len * kCommonTile + kItemCost;
            // no CTA idle; and the last common run, which is drawn after three quarters of the
            // own ones and what goes beside them
            const float all = items * item, beside = __fdividef(all, all + own_cost + 1.f) * own_cost;
            constexpr float kEach = 1.f / kSms;
            float cost = fmaxf((all + own_cost) * kEach, 0.75f * (own_cost + beside) * kEach +
                                                             ceilf(items * kEach) * item);
            // parts: written once, read once, by all rows
            cost += members * rcp * a.Hq * a.D * (4 / kPartBytes);
            if (cost < best && members * rcp <= (float)a.common_budget) {
                best = cost;
                chosen = len;
            }
        }
        const float least = __uint_as_float(__reduce_min_sync(~0u, __float_as_uint(best)));
        chosen = __shfl_sync(~0u, chosen, __ffs(__ballot_sync(~0u, best == least)) - 1);
        // never more parts than there is room for
        const float least_len = ceilf(__fdividef(members, (float)a.common_budget) * (1 + 0x1p-20f));
        chosen = max(chosen, (int32_t)fminf(least_len, (float)longest));
        chosen = max(1, min(chosen, longest));       // one run a group at most
        if (tid == 0) {
            run_len[0] = chosen;
            run_len[1] = own;
        }
    }
    __syncthreads();
    const int32_t common = run_len[0], own = run_len[1];
    const RunLength by_common(common), by_own(own);

    // ---- places: each group's first record; each sequence's first part and first record
    auto records_of = [&](const Group& x) {
        return x.keys > 0 ? row_tiles(a, x.seqs) * by_common.runs(key_tiles(a, 0, x.keys)) : 0;
    };
    auto places_of = [&](const Sequence& s) {
        const int32_t n = by_own.runs(key_tiles(a, s.prefix, s.ctx));
        return (int64_t)(n + by_common.runs(key_tiles(a, 0, s.prefix))) << 32 | n;
    };
    int64_t common_total = 0, total = 0, my_common = 0, my_place = 0;
    int64_t common_after = 0, after = 0;     // those of the first round
#pragma unroll 1
    for (int32_t base = 0; base < groups; base += threads) {
        const int64_t at = block_prefix(
            base + my_group < groups ? records_of(of.at(base + my_group, false)) : 0, common_total,
            scratch);
        if (base == 0) {
            my_common = at;
            common_after = common_total;
        }
    }
#pragma unroll 1
    for (int32_t base = 0; base < a.B; base += threads) {
        const int64_t at = block_prefix(places_of(noted(base + tid)), total, scratch);
        if (base == 0) {
            my_place = at;
            after = total;
        }
    }
    const int32_t n_common = (int32_t)common_total, n_own = (int32_t)total;
    const int32_t parts = (int32_t)(total >> 32);
    // cannot be otherwise: the run lengths allow for it
    const bool fits = common_total + n_own <= a.cap_records && parts <= a.cap_parts;
    if (tid == 0) {
        if (!fits) pkv::report(a.status, PKV_STATUS_WORKSPACE_OVERFLOW);
        a.ctrl[0] = fits ? n_common + n_own : 0;
        a.ctrl[1] = 0;
        a.part_prefix[a.B] = fits ? parts : 0;
    }
    if (!fits) {
#pragma unroll 1
        for (int32_t b = tid; b < a.B; b += threads) a.part_prefix[b] = 0;
        return;
    }
    // ---- records: each common one before `stride` own ones, over the first three quarters of
    // those, so that the two kinds run side by side and short items come last.  Many records
    // of one group or sequence are written by its warp together.
    const int32_t stride = max(1, (n_own - n_own / 4) / max(1, n_common));
#pragma unroll 1
    for (int32_t base = 0; base < groups; base += threads) {
        const int32_t g = base + my_group;
        Group x{};
        if (g < groups) x = of.at(g, false);
        const int32_t n = records_of(x);
        const int64_t place = base == 0 ? my_common : block_prefix(n, common_after, scratch);
        const int32_t from = x.keys > 0 ? table[staged ? g : x.first] : 0;
#pragma unroll 1
        for (uint32_t left = __ballot_sync(~0u, n > 0); left; left &= left - 1) {
            const int o = __ffs(left) - 1;
            const int32_t first = __shfl_sync(~0u, x.first, o), seqs = __shfl_sync(~0u, x.seqs, o);
            const int32_t keys = __shfl_sync(~0u, x.keys, o), count = __shfl_sync(~0u, n, o);
            const int32_t at0 = (int32_t)__shfl_sync(~0u, place, o);
            const int32_t src = __shfl_sync(~0u, from, o);
            const int32_t tiles = row_tiles(a, seqs), all = key_tiles(a, 0, keys);
#pragma unroll 1
            for (int32_t i = lane; i < count; i += 32) {
                const int32_t cut = i / tiles, tile = i - cut * tiles;
                Record r{};
                r.b0 = first + tile * a.tile_seqs;
                r.seqs = min(a.tile_seqs, first + seqs - r.b0);
                r.table = src;
                r.key_lo = cut * common * a.tile_keys;
                r.key_hi = (cut + 1) * common >= all ? keys : (cut + 1) * common * a.tile_keys;
                r.part = cut;
                r.origin = r.key_lo;
                // no member has keys: nobody's table to read
                r.tiles = src == INT32_MAX ? 0 : min(common, all - cut * common);
                const int64_t at = at0 + i;
                a.records[at + min(at * stride, (int64_t)n_own)] = r;
            }
        }
    }
#pragma unroll 1
    for (int32_t base = 0; base < a.B; base += threads) {
        const int32_t b = base + tid;
        const Sequence s = noted(b);
        const int64_t place = base == 0 ? my_place : block_prefix(places_of(s), after, scratch);
        if (b < a.B) a.part_prefix[b] = (int32_t)(place >> 32);
        const int32_t all = key_tiles(a, s.prefix, s.ctx), n = by_own.runs(all);
        const int32_t before = by_common.runs(key_tiles(a, 0, s.prefix));
        const int32_t origin = tile_origin(a, s.prefix);
        // a sequence of up to eight records is written by its thread, then each of the others by
        // the warp together
        uint32_t left = __ballot_sync(~0u, n > 8);
        int32_t owner = b, ctx = s.ctx, lo = s.prefix, from = origin, part = before, tiles = all;
        int32_t at = (int32_t)place, i = 0, step = 1, count = n > 8 ? 0 : n;
#pragma unroll 1
        for (;;) {
#pragma unroll 1
            for (; i < count; i += step) {
                Record r{};
                r.b0 = r.table = owner;
                r.seqs = 1;
                r.origin = from + i * own * a.tile_keys;
                r.key_lo = i == 0 ? lo : r.origin;
                r.key_hi = (i + 1) * own >= tiles ? ctx : r.origin + own * a.tile_keys;
                r.part = part + i;
                r.tiles = min(own, tiles - i * own);
                const int32_t j = at + i;
                a.records[j + min(j / stride + 1, n_common)] = r;
            }
            if (left == 0) break;
            const int o = __ffs(left) - 1;
            left &= left - 1;
            owner = __shfl_sync(~0u, b, o);
            ctx = __shfl_sync(~0u, s.ctx, o);
            lo = __shfl_sync(~0u, s.prefix, o);
            from = __shfl_sync(~0u, origin, o);
            part = __shfl_sync(~0u, before, o);
            tiles = __shfl_sync(~0u, all, o);
            at = __shfl_sync(~0u, (int32_t)place, o);
            count = __shfl_sync(~0u, n, o);
            i = lane;
            step = 32;
        }
    }
}

// ----------------------------------------------------------------- attention
template <int D>
struct __align__(1024) Smem {
    static constexpr int kTile = kKeys * D * 2;            // bytes of a Q, K or V tile
    unsigned char q[kTile];
    unsigned char k[kStages][kTile];
    unsigned char v[kStages][kTile];
    uint64_t q_full[2], q_free[2];
    uint64_t k_full[kStages], v_full[kStages], k_empty[kStages], v_empty[kStages];
    uint64_t s_full[kStages], p_full[kStages], pv_done[kStages];
    uint64_t o_free, mma_done;
    uint64_t item_full[kItemRing], item_empty[kItemRing];
    uint4 mask[kMaskRing];                                 // keys of a tile that count
    uint32_t masked_from;                                  // the first tile with a mask
    struct Item {
        int32_t b0, seqs, table, key_lo, key_hi, origin, tiles, kvh, head_tile, part;
        int32_t q_slot;                                    // half of the Q tile, 2: all of it
        int32_t end;
    } items[kItemRing];
    uint32_t tmem_base;
    int abort_flag;
};

struct Maps {
    CUtensorMap q, q_one, k, v, k_edge, v_edge;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void up2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void st_global_32b(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(saddr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(saddr(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}
__device__ __forceinline__ void cp_async16(void* smem, const void* gmem, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(saddr(smem)), "l"(gmem),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const int* abort_flag,
                                          uint32_t polls) {
    const bool r = mbar_wait(bar, parity, abort_flag, polls);
    return __all_sync(0xffffffffu, r);
}

template <class S>
__device__ __forceinline__ void give_up(S& s, uint32_t* status) {
    s.abort_flag = 1;
    pkv::report(status, PKV_STATUS_WAIT_TIMEOUT);
}

// Bit i of word i / 32: key i of a tile lies in [lo, hi).
__device__ __forceinline__ uint32_t range_word(int32_t lo, int32_t hi, int w) {
    lo = max(lo - 32 * w, 0);
    hi = min(hi - 32 * w, 32);
    if (hi <= lo) return 0;
    const uint32_t upto = hi == 32 ? ~0u : (1u << hi) - 1;
    return upto & ~((1u << lo) - 1);
}

// The K or V rows lo .. hi - 1 of a key tile by cp.async: lane l resolves rows l, l + 32, ...;
// then D / 8 lanes copy a row, each 16-byte chunk to where a 128-byte-swizzled box would put
// it.  Other rows, and those of bad blocks, are left as they are; returns whether there are such
// blocks, and the rows that were copied in `valid`.
template <int D>
__device__ __forceinline__ bool gather_rows(const SharedArgs& a, const int32_t* table,
                                            const __nv_bfloat16* pool, unsigned char* dst,
                                            int32_t key0, int32_t lo, int32_t hi, int32_t kvh,
                                            int lane, uint32_t (&valid)[4]) {
    constexpr int kChunks = D / 8, kRowsPer = 32 / kChunks;
    const int c = lane % kChunks, sub = lane / kChunks;
    bool bad = false;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int32_t i = g * 32 + lane, key = key0 + i;
        int64_t src = -1;
        if (i >= lo && i < hi) {
            const int32_t blk = __ldg(table + key / a.bs);
            if ((unsigned)blk < (unsigned)a.NB)
                src = (((int64_t)blk * a.bs + key % a.bs) * a.Hkv + kvh) * D;
            else
                bad = true;
        }
        valid[g] = __ballot_sync(0xffffffffu, src >= 0);
#pragma unroll 4
        for (int k = 0; k < 32 / kRowsPer; ++k) {
            const int rl = k * kRowsPer + sub;
            const int64_t e = __shfl_sync(0xffffffffu, src, rl);
            const int r = g * 32 + rl;
            if (e >= 0)
                cp_async16(dst + (c >> 3) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                           pool + e + c * 8, 16);
        }
    }
    return __any_sync(0xffffffffu, bad);
}

// kGather: rows gathered (block sizes that are no multiple of 8).  kPolls: the waits take
// their limit from the arguments (pkv_set_wait_poll_limit).
template <int D, bool kGather, bool kPolls>
__global__ void __launch_bounds__(kThreads, 1)
    shared_kernel(const __grid_constant__ Maps maps, const SharedArgs a) {
    using S = Smem<D>;
    using Item = typename S::Item;
    constexpr int kTile = S::kTile, kBlocks = D / 64;
    const uint32_t polls = kPolls ? a.wait_polls : (uint32_t)PKV_DEFAULT_WAIT_POLLS;
    extern __shared__ unsigned char smem_raw[];
    S& s = *reinterpret_cast<S*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        s.abort_flag = 0;
        s.masked_from = ~0u;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_free[i], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&s.k_full[i], 1);
            mbar_init(&s.v_full[i], 1);
            mbar_init(&s.k_empty[i], 1);
            mbar_init(&s.v_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 4);
            mbar_init(&s.pv_done[i], 1);
        }
        mbar_init(&s.o_free, 4);
        for (int i = 0; i < kItemRing; ++i) {
            mbar_init(&s.item_full[i], 1);
            mbar_init(&s.item_empty[i], kItemReaders);
        }
        mbar_init(&s.mma_done, 2);
        mbar_init_fence();
    }
    if (warp == 5) tmem_alloc(&s.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    pkv::wait_for_predecessor();             // the plan's records
    pkv::allow_dependent_launch();           // the combine reads the plan's parts at once
    const uint32_t units = (uint32_t)(a.Hkv * a.head_tiles);
    const uint32_t n_items = (uint32_t)a.ctrl[0] * units;
    uint32_t fills = 0;                      // a producer's tiles
    uint32_t q_uses[2] = {0, 0};             // of the halves of the Q tile

    // Item I from the ring; false: none in time.
    auto next_item = [&](uint32_t I, Item& x, bool warp_wide) {
        const int r = I % kItemRing;
        const uint32_t par = (I / kItemRing) & 1;
        const bool got = warp_wide ? warp_wait(&s.item_full[r], par, &s.abort_flag, polls)
                                   : mbar_wait(&s.item_full[r], par, &s.abort_flag, polls);
        if (!got) return false;
        x = s.items[r];
        if (warp_wide) __syncwarp();
        if (!warp_wide || lane == 0) mbar_arrive(&s.item_empty[r]);
        return true;
    };

    if (warp == 4 || warp == 7) {
        // ------------------------------------------------------------ producers
        const bool k_side = warp == 4;
        uint64_t* full_bar = k_side ? s.k_full : s.v_full;
        uint64_t* empty = k_side ? s.k_empty : s.v_empty;
        const CUtensorMap* whole_map = k_side ? &maps.k : &maps.v;
        const CUtensorMap* edge_map = k_side ? &maps.k_edge : &maps.v_edge;
        const __nv_bfloat16* pool = k_side ? a.kc : a.vc;
        if (lane == 0) {
            if (k_side) {
                tma_prefetch_desc(&maps.q);
                tma_prefetch_desc(&maps.q_one);
            }
            if (!kGather) {
                tma_prefetch_desc(whole_map);
                tma_prefetch_desc(edge_map);
            }
        }
        const uint32_t wrap = n_items + gridDim.x - 1;     // the last draw resets the counter
        auto draw = [&]() {
            return k_side && lane == 0 ? atomicInc((unsigned int*)a.ctrl + 1, wrap) : 0u;
        };
        bool ok = true, bad_block = false, masked = false;
        int q_next = 0;
        int pend = -1;                       // a gathered stage in flight
        auto land = [&](int st) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full_bar[st]);
        };
        uint32_t next = draw(), it = __shfl_sync(0xffffffffu, next, 0);
        int4 r0 = make_int4(0, 0, 0, 0);     // the record of item `it`
        int4 r1 = make_int4(0, 0, 0, 0);
        auto fetch = [&]() {
            if (it < n_items) {
                const Record* r = a.records + it / units;
                r0 = *reinterpret_cast<const int4*>(r);
                r1 = *reinterpret_cast<const int4*>(&r->key_hi);
            }
        };
        if (k_side) fetch();
        for (uint32_t I = 0; ok; ++I) {
            Item x;
            if (k_side) {
                const int ring = I % kItemRing;
                if (I >= kItemRing &&
                    !(ok = warp_wait(&s.item_empty[ring], (I / kItemRing - 1) & 1, &s.abort_flag,
                                     polls)))
                    break;
                if (it >= n_items) {
                    if (lane == 0) {
                        s.items[ring].end = 1;
                        mbar_arrive(&s.item_full[ring]);
                    }
                    break;
                }
                const uint32_t unit = it - it / units * units;
                x.b0 = r0.x;
                x.seqs = r0.y;
                x.table = r0.z;
                x.key_lo = r0.w;
                x.key_hi = r1.x;
                x.part = r1.y;
                x.origin = r1.z;
                x.tiles = r1.w;
                x.kvh = unit;
                x.head_tile = 0;
                if (a.head_tiles > 1) {
                    x.kvh = unit / a.head_tiles;
                    x.head_tile = unit - x.kvh * a.head_tiles;
                }
                x.end = 0;
                if (x.tiles == 0) next = draw();
                // the queries of one sequence take half of the Q tile, so that the next
                // item's can be loaded meanwhile
                const bool small = x.seqs == 1 && a.tile_heads <= kRows / 2;
                x.q_slot = small ? q_next : 2;
                if (x.tiles > 0 && small) q_next ^= 1;
                if (lane == 0) {
                    s.items[ring] = x;
                    mbar_arrive(&s.item_full[ring]);
                }
            } else {
                if (!(ok = next_item(I, x, true)) || x.end) break;
            }
            const int32_t* table = a.bt + (int64_t)x.table * a.MB;
            if (k_side && x.tiles > 0) {
                for (int h = 0; h < 2 && ok; ++h)
                    if ((x.q_slot == h || x.q_slot == 2) && q_uses[h] > 0)
                        ok = warp_wait(&s.q_free[h], (q_uses[h] - 1) & 1, &s.abort_flag, polls);
                if (!ok) break;
                const int first = x.q_slot == 1 ? 1 : 0;
                if (lane == 0) {
                    const CUtensorMap* m = x.seqs == 1 ? &maps.q_one : &maps.q;
                    mbar_expect_tx(&s.q_full[first],
                                   (uint32_t)(kBlocks * 128 * a.tile_heads *
                                              (x.seqs == 1 ? 1 : a.tile_seqs)));
                    for (int hf = 0; hf < kBlocks; ++hf)
                        tma_load_4d(s.q + hf * kHalf + first * (kHalf / 2), m, &s.q_full[first],
                                    hf * 64, x.head_tile * a.tile_heads, x.kvh, x.b0);
                    if (x.q_slot == 2) mbar_arrive(&s.q_full[1]);
                }
                ++q_uses[first];
                if (x.q_slot == 2) ++q_uses[1];
            }
            // Where this lane's box of a full tile is: cache block `at` of the table, row `off` of
            // it; from tile to tile without a division.
            int32_t at = 0, off = 0;
            if (!kGather) {
                const int32_t key = x.origin + lane * a.box;
                at = key / a.bs;
                off = key - at * a.bs;
            }
            for (int32_t j = 0; j < x.tiles; ++j, ++fills) {
                const int st = fills % kStages;
                const int32_t key0 = x.origin + j * a.tile_keys;
                const int32_t lo = max(x.key_lo - key0, 0), hi = min(x.key_hi - key0, a.tile_keys);
                const bool full = lo == 0 && hi == a.tile_keys;
                const int32_t box = full ? a.box : a.edge_box, i = lane * box;
                const bool wanted = !kGather && i < hi && i + box > lo;
                int32_t row = -1;
                if (wanted) {
                    int32_t block = at, r = off;
                    if (!full) {
                        block = (key0 + i) / a.bs;
                        r = key0 + i - block * a.bs;
                    }
                    const int32_t blk = __ldg(table + block);
                    if ((unsigned)blk < (unsigned)a.NB) row = blk * a.bs + r;
                }
                at += a.tile_blocks;
                off += a.tile_rest;
                if (off >= a.bs) {
                    off -= a.bs;
                    ++at;
                }
                if (k_side && j == max(x.tiles - 2, 0)) next = draw();
                if (k_side && j == x.tiles - 1) {
                    it = __shfl_sync(0xffffffffu, next, 0);
                    fetch();
                }
                const int boxes = __popc(__ballot_sync(0xffffffffu, row >= 0));
                bool bad = __any_sync(0xffffffffu, wanted && row < 0);
                if (fills >= kStages &&
                    !(ok = warp_wait(&empty[st], (fills / kStages - 1) & 1, &s.abort_flag, polls)))
                    break;
                unsigned char* dst = (k_side ? s.k[0] : s.v[0]) + st * kTile;
                uint32_t valid[4];
                if constexpr (kGather) {
                    bad = gather_rows<D>(a, table, pool, dst, key0, lo, hi, x.kvh, lane, valid);
                    asm volatile("cp.async.commit_group;" ::: "memory");
                }
                if (bad || masked) {
                    // from the first tile with a bad block on, every tile gets its mask
                    bad_block |= bad;
                    if (!kGather) {
                        const uint32_t gone = __ballot_sync(0xffffffffu, wanted && row < 0);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const int32_t k = w * 32 + lane;
                            valid[w] = __ballot_sync(
                                0xffffffffu, k >= lo && k < hi && !((gone >> (k / box)) & 1));
                        }
                    }
                    if (k_side && lane == 0) {
                        s.mask[fills % kMaskRing] =
                            make_uint4(valid[0], valid[1], valid[2], valid[3]);
                        if (!masked) *(volatile uint32_t*)&s.masked_from = fills;
                    }
                    masked = true;
                }
                if constexpr (kGather) {
                    if (pend >= 0) {         // the tile before this one has landed
                        asm volatile("cp.async.wait_group 1;" ::: "memory");
                        land(pend);
                    }
                    pend = st;
                } else {
                    if (lane == 0) {
                        if (boxes > 0)
                            mbar_expect_tx(&full_bar[st], (uint32_t)(boxes * box * 128 * kBlocks));
                        else
                            mbar_arrive(&full_bar[st]);
                    }
                    __syncwarp();
                    if (row >= 0) {
                        const CUtensorMap* m = full ? whole_map : edge_map;
                        for (int hf = 0; hf < kBlocks; ++hf)
                            tma_load_3d(dst + hf * kHalf + i * 128, m, &full_bar[st], hf * 64,
                                        x.kvh, row);
                    }
                }
            }
            if (!ok) break;
            if (k_side && x.tiles == 0) {
                it = __shfl_sync(0xffffffffu, next, 0);
                fetch();
            }
            // the next item's queries may wait for this item's last Q K^T, which waits for
            // its last K tile
            if (pend >= 0) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                land(pend);
                pend = -1;
            }
        }
        if (pend >= 0) {                     // on the way out of a wait that gave up
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            land(pend);
        }
        // every CTA draws until it gets nothing, so that the counter ends where it began
        if (k_side)
            for (it = __shfl_sync(0xffffffffu, next, 0); it < n_items;)
                it = __shfl_sync(0xffffffffu, draw(), 0);
        if (bad_block && lane == 0)
            pkv::report(a.status, PKV_STATUS_BAD_BLOCK_ID);
        if (!ok && lane == 0) give_up(s, a.status);
    } else if (warp == 5 || warp == 6) {
        // ------------------------------------------------------------ MMA issuers
        if (lane == 0) {
            const uint32_t id_qk = umma_idesc_bf16(kRows, kKeys, false);
            const uint32_t id_pv = umma_idesc_bf16(kRows, D, true);
            const uint64_t qd0 = umma_desc_sw128(saddr(s.q), 16, 1024);
            const uint64_t kd0 = umma_desc_sw128(saddr(s.k[0]), 16, 1024);
            const uint64_t vd0 = umma_desc_sw128(saddr(s.v[0]), kHalf, 1024);
            uint32_t T = 0, uses = 0;        // tiles, items with tiles so far
            bool ok = true;
            for (uint32_t I = 0; ok; ++I) {
                Item x;
                if (!(ok = next_item(I, x, false)) || x.end) break;
                if (x.tiles == 0) continue;
                if (warp == 5) {
                    for (int h = 0; h < 2 && ok; ++h)
                        if (x.q_slot == h || x.q_slot == 2)
                            ok = mbar_wait(&s.q_full[h], q_uses[h]++ & 1, &s.abort_flag, polls);
                    if (!ok) break;
                    const uint64_t qd = qd0 + (x.q_slot == 1 ? kHalf / 2 >> 4 : 0);
                    for (int32_t j = 0; j < x.tiles; ++j) {
                        const uint32_t t = T + j;
                        const int st = t % kStages;
                        if (!(ok = mbar_wait(&s.k_full[st], (t / kStages) & 1, &s.abort_flag,
                                             polls)))
                            break;
                        // the S buffer still holds P of tile t-3 until its P V is done
                        if (t >= kStages &&
                            !(ok = mbar_wait(&s.pv_done[st], (t / kStages - 1) & 1,
                                             &s.abort_flag, polls)))
                            break;
                        tc_fence_after();
                        const uint64_t kd = kd0 + (uint64_t)(st * (kTile >> 4));
                        const uint32_t d_s = tmem + st * kKeys;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                            umma_bf16(d_s, qd + off, kd + off, id_qk, kk > 0);
                        }
                        umma_commit(&s.s_full[st]);
                        umma_commit(&s.k_empty[st]);
                    }
                    if (!ok) break;
                    for (int h = 0; h < 2; ++h)
                        if (x.q_slot == h || x.q_slot == 2) umma_commit(&s.q_free[h]);
                } else {
                    for (int32_t j = 0; j < x.tiles; ++j) {
                        const uint32_t t = T + j;
                        const int st = t % kStages;
                        if (!(ok = mbar_wait(&s.p_full[st], (t / kStages) & 1, &s.abort_flag,
                                             polls)))
                            break;
                        if (j == 0 && uses > 0 &&
                            !(ok = mbar_wait(&s.o_free, (uses - 1) & 1, &s.abort_flag, polls)))
                            break;
                        if (!(ok = mbar_wait(&s.v_full[st], (t / kStages) & 1, &s.abort_flag,
                                             polls)))
                            break;
                        tc_fence_after();
                        const uint64_t vd = vd0 + (uint64_t)(st * (kTile >> 4));
                        const uint32_t a_p = tmem + st * kKeys;
                        const uint32_t acc0 = j > 0 ? 1u : 0u;
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)
                            umma_bf16_tmem_a(tmem + kColO, a_p + kk * 8, vd + (kk * 2048 >> 4),
                                             id_pv, kk > 0 ? 1u : acc0);
                        umma_commit(&s.pv_done[st]);
                        umma_commit(&s.v_empty[st]);
                    }
                    if (!ok) break;
                }
                T += x.tiles;
                ++uses;
            }
            if (!ok) give_up(s, a.status);
            // every product of both issuers has finished before TMEM is freed
            umma_commit(&s.mma_done);
            mbar_drain(&s.mma_done, 0);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int i = tid;                                 // row = TMEM lane
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const int32_t my_seq = i / a.tile_heads, my_head = i - my_seq * a.tile_heads;
        // a maximum in units of either kind as a score
        auto in_log2 = [&](float m, float unit) {
            return unit == a.scale_log2 ? m : m * a.far_ratio;
        };
        uint32_t T = 0;
        bool ok = true;
        for (uint32_t I = 0; ok; ++I) {
            Item x;
            if (!(ok = next_item(I, x, true)) || x.end) break;
            if (x.tiles == 0) continue;
            const int32_t head = x.head_tile * a.tile_heads + my_head;
            const bool mine = my_seq < x.seqs && head < a.G;
            const bool active = warp * 32 < x.seqs * a.tile_heads;
            // asked for ahead of its use behind the tiles
            const int32_t b = x.b0 + my_seq;
            const int32_t first = mine ? a.part_prefix[b] : 0;
            const int32_t parts = mine ? a.part_prefix[b + 1] - first : 0;  // 0: without keys
            float m_run = -INFINITY, l_run = 0.f, unit = a.scale_log2;
            for (int32_t j = 0; j < x.tiles && ok; ++j) {
                const uint32_t t = T + j;
                const int st = t % kStages;
                const uint32_t s_col = lanes + st * kKeys;
                if (!(ok = warp_wait(&s.s_full[st], (t / kStages) & 1, &s.abort_flag, polls)))
                    break;
                tc_fence_after();
                // Tiles with a bad block are rare: their masks come through shared memory,
                // the others' follow from the run.  (The producer wrote them before it
                // filled the tile's K stage, which Q K^T waited for.)
                const int32_t key0 = x.origin + j * a.tile_keys;
                const int32_t lo = max(x.key_lo - key0, 0);
                const int32_t hi = min(x.key_hi - key0, a.tile_keys);
                const bool marked = t >= *(volatile uint32_t*)&s.masked_from;
                const bool whole = !marked && lo == 0 && hi == kKeys;
                uint32_t mask[4] = {~0u, ~0u, ~0u, ~0u};
                if (!whole) {
                    const uint4 mk = s.mask[t % kMaskRing];
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        mask[w] = marked ? pkv::word(mk, w) : range_word(lo, hi, w);
                }
                if (active) {
                    float sv[kKeys];
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc) tmem_ld32(s_col + cc * 32, sv + cc * 32);
                    tmem_wait_ld();
                    if (!whole) {
#pragma unroll
                        for (int c = 0; c < kKeys; ++c)
                            sv[c] = (mask[c >> 5] >> (c & 31)) & 1 ? sv[c] : -INFINITY;
                    }
                    float sum = 0.f;
                    // P against `neg_m` over the first 64 columns of S, and its sum
                    auto exp_pass = [&](float neg_m) {
                        const uint64_t scale2 = pk2(unit, unit);
                        const uint64_t neg2 = pk2(neg_m, neg_m);
                        uint64_t l2[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float pw[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const int c = half * 64 + 2 * e;
                                float x0, x1;
                                up2(fma2(pk2(sv[c], sv[c + 1]), scale2, neg2), x0, x1);
                                const float p0 = pkv::fast_exp2(x0), p1 = pkv::fast_exp2(x1);
                                l2[e & 1] = add2(l2[e & 1], pk2(p0, p1));
                                pw[e] = __uint_as_float(pkv::pack_bf16(p0, p1));
                            }
                            tmem_st32(s_col + half * 32, pw);
                        }
                        float s0, s1, s2, s3;
                        up2(l2[0], s0, s1);
                        up2(l2[1], s2, s3);
                        sum = (s0 + s1) + (s2 + s3);
                    };
                    // One pass where P stands against the running maximum; else a second,
                    // with the maximum taken first (as for an item's first tile).
                    bool take = j == 0, again;
                    do {
                        if (take) {
                            float part[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) part[e] = fmaxf(sv[e], sv[8 + e]);
#pragma unroll
                            for (int c = 16; c < kKeys; c += 16)
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    part[e] = max3(part[e], sv[c + e], sv[c + 8 + e]);
                            float mx =
                                fmaxf(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])),
                                      fmaxf(fmaxf(part[4], part[5]), fmaxf(part[6], part[7])));
                            const float score = mx * a.scale_log2;    // scale > 0 keeps the order
                            const float u =
                                fabsf(score) >= pkv::kFarScore ? a.far_unit : a.scale_log2;
                            mx *= u;
                            const bool raise =
                                mine && (u == unit ? mx > m_run - (kHeadroom - kRescaleThreshold)
                                                   : score > in_log2(m_run, unit));
                            float alpha = 1.f;
                            if (raise) {
                                // (maxima of different units are far apart)
                                alpha = m_run == -INFINITY || u != unit
                                            ? 0.f
                                            : pkv::fast_exp2(m_run - (mx + kHeadroom));
                                m_run = mx + kHeadroom;
                                unit = u;
                                // a score that 32 bits do not hold: the row is NaN
                                l_run *= score < INFINITY ? alpha : NAN;
                            }
                            if (j > 0 && __any_sync(0xffffffffu, raise)) {
                                // O may only be rescaled once the last P V has finished
                                const uint32_t tp = t - 1;
                                if (!(ok = warp_wait(&s.pv_done[tp % kStages], (tp / kStages) & 1,
                                                     &s.abort_flag, polls)))
                                    break;
                                tc_fence_after();
#pragma unroll 1
                                for (int cc = 0; cc < D / 32; ++cc) {
                                    float ov[32];
                                    tmem_ld32(lanes + kColO + cc * 32, ov);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; ++e) ov[e] *= alpha;
                                    tmem_st32(lanes + kColO + cc * 32, ov);
                                }
                            }
                        }
                        // (without a maximum yet, the sum is infinite or NaN the first time)
                        exp_pass(take && m_run == -INFINITY ? 0.f : -m_run);
                        again = !take && __any_sync(0xffffffffu, mine && !(sum <= kSumTrigger));
                        take = again;
                        if (again) tmem_wait_st();         // before P is stored again
                    } while (again);
                    if (!ok) break;
                    l_run += sum;
                    tmem_wait_st();
                }
                if (!whole) {
                    // V rows of keys that do not count may hold anything: thread i clears row i
                    if (!(ok = warp_wait(&s.v_full[st], (t / kStages) & 1, &s.abort_flag, polls)))
                        break;
                    if (!((mask[warp] >> lane) & 1)) {
#pragma unroll
                        for (int hf = 0; hf < kBlocks; ++hf)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                *reinterpret_cast<uint4*>(s.v[st] + hf * kHalf + i * 128 + c * 16) =
                                    make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.p_full[st]);
            }
            if (!ok) break;
            // ---- this item's part, or the result where there is no other
            T += x.tiles;
            if (!(ok = warp_wait(&s.pv_done[(T - 1) % kStages], ((T - 1) / kStages) & 1,
                                 &s.abort_flag, polls)))
                break;
            tc_fence_after();
            if (active) {
                const int64_t row = x.kvh * a.G + head;
                const int64_t at = ((int64_t)first + x.part) * a.Hq + row;
                const bool some = l_run > 0.f || l_run != l_run;
                const float inv = some ? 1.f / l_run : 0.f;
                const bool wide = ((uintptr_t)a.out & 31) == 0;
                __nv_bfloat16* out = a.out + ((int64_t)b * a.Hq + row) * D;
#pragma unroll 1
                for (int cc = 0; cc < D / 32; ++cc) {
                    float ov[32];
                    tmem_ld32(lanes + kColO + cc * 32, ov);
                    tmem_wait_ld();
                    if (parts > 1) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) w[k] = __float_as_uint(ov[e + k]);
                            st_global_32b(a.part_o + at * D + cc * 32 + e, w);
                        }
                    } else if (parts == 1) {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            uint32_t w[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                w[k] = some ? pkv::pack_bf16(ov[e + 2 * k] * inv,
                                                             ov[e + 2 * k + 1] * inv)
                                            : 0u;
                            if (wide) {
                                st_global_32b(out + cc * 32 + e, w);
                            } else {
                                uint4* to = reinterpret_cast<uint4*>(out + cc * 32 + e);
                                to[0] = make_uint4(w[0], w[1], w[2], w[3]);
                                to[1] = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    }
                }
                if (parts > 1) a.part_ml[at] = make_float2(0.5f * in_log2(m_run, unit), l_run);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.o_free);
        }
        if (!ok && lane == 0) give_up(s, a.status);
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (s.abort_flag && lane == 0 && (warp == 4 || warp == 7)) {
        // some role gave up: every copy this producer issued lands before the CTA exits
        for (uint32_t back = 1; back <= (uint32_t)kStages && back <= fills; ++back) {
            const uint32_t f = fills - back;
            mbar_drain(warp == 4 ? &s.k_full[f % kStages] : &s.v_full[f % kStages],
                       (f / kStages) & 1);
        }
        if (warp == 4)
            for (int h = 0; h < 2; ++h)
                if (q_uses[h] > 0) mbar_drain(&s.q_full[h], (q_uses[h] - 1) & 1);
    }
    if (warp == 5) tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------------- host
struct Layout {
    int32_t box, edge_box, tile_keys, tile_heads, head_tiles, tile_seqs;
    int32_t cap_records, cap_parts, common_budget;
    size_t off_prefix, off_sequences, off_table, off_records, off_ml, off_o, total;
};

// Rows of a TMA box: a run of a cache block (a multiple of 8 rows, what the swizzle
// repeats after).  Of those of 16 rows or more the one that fills most of a 128-key tile,
// the largest of several; 8 where there is none.  Block sizes that are no multiple of 8
// are gathered row by row (box 1).
int32_t choose_box(int32_t bs) {
    if (bs % 8 != 0) return 1;
    int32_t best = 8, fill = 0;
    for (int32_t box = 16; box <= kKeys && box <= bs; box += 8) {
        if (bs % box != 0) continue;
        const int32_t keys = kKeys / box * box;
        if (keys >= fill) {
            best = box;
            fill = keys;
        }
    }
    return best;
}

bool layout(int32_t batch, int32_t num_q_heads, int32_t max_ctx, const pkv_cache_desc& c,
            Layout& L) {
    L = Layout{};
    const int32_t G = num_q_heads / c.num_kv_heads;
    L.box = choose_box(c.block_size);
    L.edge_box = L.box % 16 == 0 ? 16 : L.box;
    if (L.box % 16 != 0 && L.box > 8) L.edge_box = 8;
    L.tile_keys = kKeys / L.box * L.box;
    L.tile_heads = G < kRows ? G : kRows;
    L.head_tiles = ceil_div(G, L.tile_heads);
    L.tile_seqs = kRows / L.tile_heads;
    // Parts, one of a run for each of its sequences.  Own runs are long enough for 16 kSms
    // items in all, and one more for each sequence; common runs, so long that their items
    // could be 8 kSms of tile_seqs sequences each, and one more for each sequence.  Neither
    // is more than the tiles there can be.
    const int64_t units = (int64_t)c.num_kv_heads * L.head_tiles;
    if (max_ctx > kMaxContext) return false;
    const int64_t tiles = (int64_t)batch * (ceil_div(max_ctx, L.tile_keys) + 1);
    const int64_t own = (16 * kSms + units - 1) / units;
    const int64_t common = ((int64_t)L.tile_seqs * 8 * kSms + units - 1) / units;
    L.common_budget = (int32_t)(common < tiles ? common : tiles);
    if (L.common_budget < 1) L.common_budget = 1;
    const int64_t parts = L.common_budget + (own < tiles ? own : tiles) + 2 * (int64_t)batch + 2;
    if (parts > (1 << 30) || parts * units >= (1LL << 31)) return false;
    L.cap_parts = L.cap_records = (int32_t)parts;
    auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
    L.off_prefix = 256;
    L.off_sequences = align(L.off_prefix + sizeof(int32_t) * ((size_t)batch + 1));
    L.off_table = align(L.off_sequences + sizeof(int2) * (size_t)batch);
    L.off_records = align(L.off_table + sizeof(int32_t) * (size_t)batch);
    L.off_ml = align(L.off_records + sizeof(Record) * (size_t)L.cap_records);
    L.off_o = align(L.off_ml + sizeof(float2) * (size_t)L.cap_parts * num_q_heads);
    L.total = align(L.off_o + sizeof(float) * (size_t)L.cap_parts * num_q_heads * c.head_dim);
    L.total += 256;                          // the workspace is 16-byte aligned, parts by 256
    return true;
}


// Checks what the plan depends on and fills its part of `a`.
int make_plan(int32_t batch, int32_t num_q_heads, int32_t max_context_len,
              int32_t max_blocks_per_seq, void* workspace, size_t workspace_bytes,
              const pkv_cache_desc& cache, uint32_t* status, SharedArgs& a) {
    if (batch < 0 || max_context_len < 0 || max_blocks_per_seq <= 0 || num_q_heads <= 0 ||
        cache.num_blocks <= 0 || cache.block_size <= 0 || cache.num_kv_heads <= 0)
        return PKV_ERR_BAD_DIMENSION;
    if (num_q_heads % cache.num_kv_heads != 0) return PKV_ERR_BAD_DIMENSION;
    if (cache.head_dim != 64 && cache.head_dim != 128) return PKV_ERR_UNSUPPORTED_HEAD_DIM;
    if ((int64_t)cache.num_blocks * cache.block_size >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;
    // (first, for there is no workspace of such sizes: the query gives 0)
    Layout L;
    if (!layout(batch, num_q_heads, max_context_len, cache, L)) return PKV_ERR_UNSUPPORTED;
    if (!workspace) return PKV_ERR_NULL_POINTER;
    if ((uintptr_t)workspace & 15) return PKV_ERR_MISALIGNED;
    if (workspace_bytes < L.total) return PKV_ERR_WORKSPACE_TOO_SMALL;
    char* ws = (char*)(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    a = SharedArgs{};
    a.ctrl = (int32_t*)ws;
    a.part_prefix = (int32_t*)(ws + L.off_prefix);
    a.sequences = (int2*)(ws + L.off_sequences);
    a.table = (int32_t*)(ws + L.off_table);
    a.records = (Record*)(ws + L.off_records);
    a.part_ml = (float2*)(ws + L.off_ml);
    a.part_o = (float*)(ws + L.off_o);
    a.B = batch;
    a.Hq = num_q_heads;
    a.Hkv = cache.num_kv_heads;
    a.G = num_q_heads / cache.num_kv_heads;
    a.MB = max_blocks_per_seq;
    a.NB = cache.num_blocks;
    a.bs = cache.block_size;
    a.D = cache.head_dim;
    a.max_ctx = max_context_len;
    a.box = L.box;
    a.edge_box = L.edge_box;
    a.tile_keys = L.tile_keys;
    a.tile_blocks = L.tile_keys / cache.block_size;
    a.tile_rest = L.tile_keys % cache.block_size;
    a.tile_heads = L.tile_heads;
    a.head_tiles = L.head_tiles;
    a.tile_seqs = L.tile_seqs;
    a.cap_records = L.cap_records;
    a.cap_parts = L.cap_parts;
    a.common_budget = L.common_budget;
    a.status = status;
    a.wait_polls = pkv_wait_polls();
    auto divisor = [](int32_t d) {
        int32_t l = 0;
        while ((1 << l) < d) ++l;
        return Divisor{(uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
    };
    a.by_box = divisor(a.box);
    a.by_tile = divisor(a.tile_keys);
    a.by_seqs = divisor(a.tile_seqs);
    return PKV_OK;
}

int add_lengths(const int32_t* context_lens, const int32_t* group_offsets,
                const int32_t* prefix_lens, int32_t num_groups, SharedArgs& a) {
    if (num_groups < 0) return PKV_ERR_BAD_DIMENSION;
    if (!context_lens || (num_groups > 0 && (!group_offsets || !prefix_lens)))
        return PKV_ERR_NULL_POINTER;
    if (((uintptr_t)context_lens | (uintptr_t)group_offsets | (uintptr_t)prefix_lens) & 3)
        return PKV_ERR_MISALIGNED;
    a.ctx = context_lens;
    a.offsets = group_offsets;
    a.prefix = prefix_lens;
    a.groups = num_groups;
    return PKV_OK;
}

int add_tensors(const void* q, const void* k_cache, const void* v_cache,
                const int32_t* block_tables, float scale, void* out, SharedArgs& a) {
    if (!(scale > 0.f) || !isfinite(scale)) return PKV_ERR_BAD_DIMENSION;
    if (!q || !k_cache || !v_cache || !block_tables || !out) return PKV_ERR_NULL_POINTER;
    if (((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out) & 15)
        return PKV_ERR_MISALIGNED;
    if ((uintptr_t)block_tables & 3) return PKV_ERR_MISALIGNED;
    if (pkv::tma_encode_fn() == nullptr) return PKV_ERR_UNSUPPORTED;
    a.q = (const __nv_bfloat16*)q;
    a.kc = (const __nv_bfloat16*)k_cache;
    a.vc = (const __nv_bfloat16*)v_cache;
    a.bt = block_tables;
    a.out = (__nv_bfloat16*)out;
    a.scale_log2 = scale * pkv::kLog2e;
    a.far_unit = pkv::power_below(a.scale_log2);
    a.far_ratio = a.scale_log2 / a.far_unit;
    return PKV_OK;
}

int launch_plan(const SharedArgs& a, cudaStream_t s) {
    plan_kernel<<<1, a.B <= 256 ? 256 : a.B <= 512 ? 512 : kMaxPlanThreads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// q as [batch, Hkv, G, D]; a box is 64 entries of tile_heads heads of `seqs` sequences, so
// that its rows are the sequences' heads in turn.
bool encode_q(CUtensorMap* m, const SharedArgs& a, int32_t seqs) {
    const cuuint64_t D = (cuuint64_t)a.D;
    cuuint64_t dims[4] = {D, (cuuint64_t)a.G, (cuuint64_t)a.Hkv, (cuuint64_t)a.B};
    cuuint64_t strides[3] = {D * 2, D * 2 * a.G, D * 2 * a.Hq};
    cuuint32_t box[4] = {64, (cuuint32_t)a.tile_heads, 1, (cuuint32_t)seqs};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return pkv::tma_encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, (void*)a.q, dims, strides,
                                box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_maps(const SharedArgs& a, Maps& m) {
    if (!encode_q(&m.q, a, a.tile_seqs) || !encode_q(&m.q_one, a, 1)) return false;
    m.k = m.v = m.k_edge = m.v_edge = m.q;   // not used where rows are gathered
    if (a.box == 1) return true;
    const int64_t rows = (int64_t)a.NB * a.bs;
    return pkv::tma_encode_rows(&m.k, a.kc, rows, a.Hkv, a.D, a.box) &&
           pkv::tma_encode_rows(&m.v, a.vc, rows, a.Hkv, a.D, a.box) &&
           pkv::tma_encode_rows(&m.k_edge, a.kc, rows, a.Hkv, a.D, a.edge_box) &&
           pkv::tma_encode_rows(&m.v_edge, a.vc, rows, a.Hkv, a.D, a.edge_box);
}

template <int D>
int launch_attention(const SharedArgs& a, const Maps& maps, cudaStream_t s) {
    using Kernel = void (*)(const Maps, const SharedArgs);
    static const Kernel kernels[4] = {shared_kernel<D, false, false>, shared_kernel<D, false, true>,
                                      shared_kernel<D, true, false>, shared_kernel<D, true, true>};
    static std::atomic<uint64_t> configured[4];
    const int which = (a.box == 1 ? 2 : 0) +
                      (a.wait_polls != (uint32_t)PKV_DEFAULT_WAIT_POLLS ? 1 : 0);
    const int smem = (int)sizeof(Smem<D>) + 1024;
    if (!pkv_dynamic_smem_once((const void*)kernels[which], smem, configured[which]))
        return PKV_ERR_CUDA;
    int64_t grid = pkv_num_sms();
    const int64_t upper = (int64_t)a.cap_records * a.Hkv * a.head_tiles;
    if (grid > upper) grid = upper;
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
    if (cudaLaunchKernelEx(&cfg, kernels[which], maps, a) != cudaSuccess) return PKV_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// The attention and the combine of the sequences' parts (that of the e4m3 decode: maxima
// halved, NaN kept).
int launch_run(const SharedArgs& a, const Maps& maps, cudaStream_t s) {
    const int rc = a.D == 128 ? launch_attention<128>(a, maps, s)
                              : launch_attention<64>(a, maps, s);
    if (rc != PKV_OK) return rc;
    pkv::DecodeArgs d{};
    d.out = a.out;
    d.chunk_prefix = a.part_prefix;
    d.part_ml = a.part_ml;
    d.part_o = a.part_o;
    d.B = a.B;
    d.Hq = a.Hq;
    return pkv_launch_decode_combine(d, a.D, s);
}

}  // namespace

extern "C" size_t pkv_paged_decode_shared_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                                          int32_t max_context_len,
                                                          pkv_cache_desc cache) {
    if (batch < 0 || num_q_heads <= 0 || max_context_len < 0 || cache.num_kv_heads <= 0 ||
        cache.block_size <= 0 || cache.head_dim <= 0 || num_q_heads % cache.num_kv_heads != 0)
        return 0;
    Layout L;
    return layout(batch, num_q_heads, max_context_len, cache, L) ? L.total : 0;
}

extern "C" int pkv_paged_decode_plan_shared(const int32_t* context_lens,
                                            const int32_t* group_offsets,
                                            const int32_t* prefix_lens, int32_t num_groups,
                                            int32_t batch, int32_t num_q_heads,
                                            int32_t max_context_len, int32_t max_blocks_per_seq,
                                            void* workspace, size_t workspace_bytes,
                                            pkv_cache_desc cache, uint32_t* status, void* stream) {
    if (batch == 0 && max_context_len >= 0 && num_q_heads > 0) return PKV_OK;
    SharedArgs a;
    int rc = make_plan(batch, num_q_heads, max_context_len, max_blocks_per_seq, workspace,
                       workspace_bytes, cache, status, a);
    if (rc == PKV_OK) rc = add_lengths(context_lens, group_offsets, prefix_lens, num_groups, a);
    return rc == PKV_OK ? launch_plan(a, (cudaStream_t)stream) : rc;
}

extern "C" int pkv_paged_decode_run_shared(const void* q, const void* k_cache,
                                           const void* v_cache, const int32_t* block_tables,
                                           int32_t max_blocks_per_seq, int32_t batch,
                                           int32_t num_q_heads, int32_t max_context_len,
                                           float scale, void* out, void* workspace,
                                           size_t workspace_bytes, pkv_cache_desc cache,
                                           uint32_t* status, void* stream) {
    if (batch == 0 && max_context_len >= 0 && num_q_heads > 0) return PKV_OK;
    SharedArgs a;
    int rc = make_plan(batch, num_q_heads, max_context_len, max_blocks_per_seq, workspace,
                       workspace_bytes, cache, status, a);
    if (rc == PKV_OK) rc = add_tensors(q, k_cache, v_cache, block_tables, scale, out, a);
    if (rc != PKV_OK) return rc;
    Maps maps;
    if (!encode_maps(a, maps)) return PKV_ERR_CUDA;
    return launch_run(a, maps, (cudaStream_t)stream);
}

extern "C" int pkv_paged_decode_shared(const void* q, const void* k_cache, const void* v_cache,
                                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                                       const int32_t* context_lens, const int32_t* group_offsets,
                                       const int32_t* prefix_lens, int32_t num_groups,
                                       int32_t batch, int32_t num_q_heads,
                                       int32_t max_context_len, float scale, void* out,
                                       void* workspace, size_t workspace_bytes,
                                       pkv_cache_desc cache, uint32_t* status, void* stream) {
    if (batch == 0 && max_context_len >= 0 && num_q_heads > 0) return PKV_OK;
    SharedArgs a;
    int rc = make_plan(batch, num_q_heads, max_context_len, max_blocks_per_seq, workspace,
                       workspace_bytes, cache, status, a);
    if (rc == PKV_OK) rc = add_lengths(context_lens, group_offsets, prefix_lens, num_groups, a);
    if (rc == PKV_OK) rc = add_tensors(q, k_cache, v_cache, block_tables, scale, out, a);
    if (rc != PKV_OK) return rc;
    Maps maps;
    if (!encode_maps(a, maps)) return PKV_ERR_CUDA;
    rc = launch_plan(a, (cudaStream_t)stream);
    return rc == PKV_OK ? launch_run(a, maps, (cudaStream_t)stream) : rc;
}
