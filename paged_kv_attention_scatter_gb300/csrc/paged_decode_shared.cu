// paged_decode_shared: decode attention for a batch whose sequences come in groups with
// their first keys in common (one system prompt, one document, several samples of one
// prompt), the common keys read and multiplied once for all sequences of a group.
//
// What it computes: what paged_decode does,
//   out[b,h] = sum_{j < ctx_b} softmax_j(scale * q[b,h] . K_j) V_j.
// For a group of n sequences with P common keys the queries of one kv head are the
// n G rows of a matrix, so that Q K^T and P V over the common keys are matrix products
// of n G rows on the tensor cores, and the K and V rows are read once, not n times.  The
// softmax over a sequence's keys is put together from parts: each part is a maximum m, a
// sum l and an unnormalised o over some of the keys, and
//   M = max m,  out = sum 2^(m - M) o / sum 2^(m - M) l.
//
// Work item = (record, kv head, tile of q heads).  A record is a run of keys for up to 256
// rows: either common keys of a group's sequences, or own keys of one sequence.  Both go
// through the same kernel, so that items bound by the tensor cores (many rows on the same
// keys) and items bound by HBM (a few rows on keys of their own) run side by side.  One CTA
// of plan_kernel sizes the records from the lengths and lays them out; CTAs of the
// persistent attention kernel, one an SM, draw items from a counter.
//
// A CTA attends 128-row tiles against 128-key tiles:
//   warps 0-3, 4-7  two softmax groups; thread i of a group owns row i = TMEM lane i.
//                   P = exp2(S scale - m) is computed against the running maximum straight
//                   away, and again, with the maximum taken and O and l rescaled, only
//                   where its row sum passes 2^16 (and for the first tile).  P stays in
//                   registers until then and goes over S in TMEM as bf16, unnormalised:
//                   its relative rounding of 2^-9 is that of a bf16 softmax, l is summed
//                   from the unrounded values.
//   warp 8          the producer: draws items, loads Q tiles, K and V tiles (TMA, one box per
//                   run of a cache block, or rows gathered with cp.async where the block
//                   size is no multiple of 8)
//   warp 9, 10      issue Q K^T and P V (tcgen05.mma, accumulators in TMEM)
// An item of two row tiles gives each group its own: both multiply the same K and V
// tiles, which halves what is read from L2 for each product.  An item of one row tile has
// its key tiles dealt to the two groups in turn, each with a maximum, sum and O of its
// own (two parts), so that one group's softmax runs beside the other's products.
// TMEM columns: S0 [0,128), S1 [128,256), O0 [256,256+D), O1 [384,384+D).
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
constexpr int kThreads = 384;
constexpr int kItemRing = 4, kItemReaders = 10;
constexpr int kMaskRing = 16;            // more tiles than are between producer and softmax
constexpr float kRescaleThreshold = 8.0f;   // log2 of the tolerated growth of a maximum
constexpr float kSumTrigger = 65536.0f;
constexpr int kSms = 152;                // of a GB300: sizes follow from the arguments alone

// A run of keys for `seqs` sequences from b0 on (1: own keys of b0, read through its own
// table; more: common keys, read through that of sequence `table`).
struct Record {
    int32_t b0, seqs, table, key_lo, key_hi;
    int32_t part;                        // place of its (first) part among a sequence's
    int32_t pad0, pad1;
};

struct SharedArgs {
    const __nv_bfloat16* q;
    const __nv_bfloat16* kc;
    const __nv_bfloat16* vc;
    const int32_t* bt;
    __nv_bfloat16* out;
    int32_t* ctrl;                       // [0] records, [1] items drawn
    int32_t* part_prefix;                // [B + 1]: parts of the sequences before
    int32_t* group;                      // [B]: the sequence's group, -1: none
    int32_t* table;                      // [B], at a group's first sequence: whose table
    Record* records;
    float2* part_ml;                     // [cap_parts, Hq]: (max halved, sum)
    float* part_o;                       // [cap_parts, Hq, D]
    int32_t B, Hq, Hkv, G, MB, NB, bs, max_ctx, D;
    int32_t box, edge_box, tile_keys;    // rows of a TMA box; in tiles not full; keys of a tile
    int32_t tile_heads, head_tiles, tile_seqs;
    int32_t cap_records, cap_parts, common_budget;
    float scale_log2;
    uint32_t* status;
    uint32_t wait_polls;
    // the plan's
    const int32_t* ctx;
    const int32_t* offsets;
    const int32_t* prefix;
    int32_t groups;
};

__host__ __device__ __forceinline__ int32_t ceil_div(int32_t a, int32_t b) {
    return (a + b - 1) / b;
}

// ---------------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024;
// Fewer common keys than this are attended by each sequence itself.
constexpr int kMinShared = 64;
// What the plan expects, in ns: a key tile for two row tiles and for one, the start and end
// of an item, and the bytes a ns of parts written and read again.
constexpr int kPairTile = 1150, kTileCost = 1450, kItemCost = 2000, kPartBytes = 3500;

struct Group {
    int32_t first, seqs;
    int32_t prefix;                      // keys in common
    int32_t keys;                        // those attended together: all of them, or 0
};

// Group g of the call; `ok`: the offsets are increasing and within the batch.
__device__ __forceinline__ Group group_at(const SharedArgs& a, int32_t g, bool report) {
    Group x{a.offsets[g], 0, a.prefix[g], 0};
    x.seqs = a.offsets[g + 1] - x.first;
    if (x.prefix < 0 || x.prefix > (int64_t)a.MB * a.bs || x.prefix > a.max_ctx) {
        if (report) pkv::report(a.status, PKV_STATUS_BAD_SEQLENS);
        x.prefix = 0;
    }
    if (x.seqs >= 2 && x.prefix >= kMinShared) x.keys = x.prefix;
    return x;
}

// The first key tile of a run begins at a box of the cache block that key_lo lies in.
__device__ __forceinline__ int32_t tile_origin(const SharedArgs& a, int32_t key_lo) {
    return key_lo / a.box * a.box;
}
__device__ __forceinline__ int32_t key_tiles(const SharedArgs& a, int32_t lo, int32_t hi) {
    return ceil_div(hi - tile_origin(a, lo), a.tile_keys);
}

// Block-wide sum of v.
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* scratch) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(~0u, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = scratch[threadIdx.x & 31];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(~0u, v, off);
    return v;
}

// Block-wide exclusive prefix of v, over `carry` (updated to the sum).
__device__ __forceinline__ int32_t block_prefix(int32_t v, int32_t& carry, int32_t* scratch) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int32_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int32_t y = __shfl_up_sync(~0u, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch[w] = x;
    __syncthreads();
    int32_t s = scratch[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int32_t y = __shfl_up_sync(~0u, s, off);
        if (lane >= off) s += y;
    }
    const int32_t before = w > 0 ? __shfl_sync(~0u, s, w - 1) : 0;
    const int32_t all = __shfl_sync(~0u, s, 31);
    const int32_t r = carry + before + x - v;
    carry += all;
    return r;
}

// Parts of `tiles` key tiles cut every `len`: two of a run where its tiles are dealt to two
// softmax groups, one where each group has rows of its own.
__device__ __forceinline__ int32_t parts_of(int32_t tiles, int32_t len, bool dealt) {
    const int32_t runs = ceil_div(tiles, len);
    if (!dealt || runs == 0) return runs;
    const int32_t last = tiles - (runs - 1) * len;
    return (runs - 1) * min(2, len) + min(2, last);
}

// What a sequence attends: keys [0, prefix) with its group, [prefix, ctx) on its own.
struct Sequence {
    int32_t ctx, prefix, own_tiles;
    bool dealt;                          // its row tile is the last, without another beside it
    int32_t prefix_tiles;
};

__device__ __forceinline__ Sequence sequence_at(const SharedArgs& a, int32_t b, bool report) {
    Sequence s{0, 0, 0, true, 0};
    int32_t c = a.ctx[b];
    if (c < 0 || c > (int64_t)a.MB * a.bs || c > a.max_ctx) {
        if (report) pkv::report(a.status, PKV_STATUS_BAD_CONTEXT_LEN);
        return s;
    }
    if (c == 0) return s;
    const int32_t g = a.group[b];
    if (g >= 0) {
        const Group x = group_at(a, g, false);
        if (x.prefix > c) {                  // a member without all of its group's keys
            if (report) pkv::report(a.status, PKV_STATUS_BAD_CONTEXT_LEN);
            return s;
        }
        if (x.keys > 0) {
            s.prefix = x.keys;
            s.prefix_tiles = key_tiles(a, 0, x.keys);
            const int32_t tiles = ceil_div(x.seqs, a.tile_seqs);
            s.dealt = (tiles & 1) && (b - x.first) / a.tile_seqs == tiles - 1;
        }
    }
    s.ctx = c;
    s.own_tiles = c > s.prefix ? key_tiles(a, s.prefix, c) : 0;
    return s;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(SharedArgs a) {
    pkv::allow_dependent_launch();
    __shared__ int64_t sums[32];
    __shared__ int32_t scans[32];
    __shared__ int32_t run_len[2];           // key tiles of a common run, of an own run
    const int tid = threadIdx.x;
    const int32_t units = a.Hkv * a.head_tiles;

    // ---- groups: increasing offsets within the batch, or none is used
    bool bad = false;
    for (int32_t g = tid; g <= a.groups; g += kPlanThreads) {
        const int32_t o = a.groups > 0 ? a.offsets[g] : 0;
        bad |= o < 0 || o > a.B || (g > 0 && o < a.offsets[g - 1]);
    }
    const int32_t groups = __syncthreads_or(bad) ? 0 : a.groups;
    if (groups != a.groups && tid == 0) pkv::report(a.status, PKV_STATUS_BAD_SEQLENS);
    for (int32_t b = tid; b < a.B; b += kPlanThreads) {
        int32_t lo = 0, hi = groups;         // groups that begin at b or before
        while (lo < hi) {
            const int32_t mid = (lo + hi) / 2;
            if (a.offsets[mid] <= b) lo = mid + 1;
            else hi = mid;
        }
        a.group[b] = lo > 0 && b < a.offsets[lo] ? lo - 1 : -1;
        a.table[b] = INT32_MAX;
    }
    __syncthreads();
    // ---- how much there is: common tiles of row pairs and of lone row tiles, own tiles
    int64_t pair_tiles = 0, lone_tiles = 0, own_tiles = 0, members = 0, runs = 0;
    for (int32_t g = tid; g < groups; g += kPlanThreads) {
        const Group x = group_at(a, g, true);
        if (x.keys == 0) continue;
        const int32_t tiles = ceil_div(x.seqs, a.tile_seqs), n = key_tiles(a, 0, x.keys);
        pair_tiles += (int64_t)(tiles / 2) * n;
        lone_tiles += (int64_t)(tiles & 1) * n;
        runs += (tiles + 1) / 2;
        members += (int64_t)x.seqs * n;
    }
    int32_t busy = 0;
    for (int32_t b = tid; b < a.B; b += kPlanThreads) {
        const Sequence s = sequence_at(a, b, true);
        own_tiles += s.own_tiles;
        busy += s.own_tiles > 0;
        if (s.prefix > 0) atomicMin(&a.table[a.offsets[a.group[b]]], b);
    }
    pair_tiles = block_sum(pair_tiles, sums);
    lone_tiles = block_sum(lone_tiles, sums);
    own_tiles = block_sum(own_tiles, sums);
    members = block_sum(members, sums);
    runs = block_sum(runs, sums);
    const int32_t sequences = (int32_t)block_sum(busy, sums);

    // ---- run lengths: lane l of the first warp weighs common runs of a length
    if (tid < 32) {
        // own runs: eight items an SM up to four tiles each, then up to sixteen items
        const int64_t eight = (own_tiles * units + 8 * kSms - 1) / (8 * kSms);
        const int64_t sixteen = (own_tiles * units + 16 * kSms - 1) / (16 * kSms);
        const int32_t own = (int32_t)max(max(min(eight, (int64_t)4), sixteen), (int64_t)1);
        const int64_t own_cost = (own_tiles * kTileCost +
                                  (own_tiles / own + sequences) * kItemCost) * units;
        // lengths 1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 14, 16, 20, ...
        const int l = tid;
        const int32_t len = l < 4 ? l + 1 : (4 + (l & 3)) << ((l >> 2) - 1);
        const int64_t items = ((pair_tiles + lone_tiles) / len + runs) * units;
        const int64_t item = (int64_t)len * (pair_tiles > 0 ? kPairTile : kTileCost) + kItemCost;
        const int64_t rounds = (items + kSms - 1) / kSms;
        int64_t cost = max(rounds * item, (items * item + own_cost) / kSms);
        // parts: written once, read once, by all rows
        cost += members / len * a.Hq * a.D * 4 / kPartBytes;
        if (members / len > a.common_budget) cost = INT64_MAX;
        int64_t best = cost;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) best = min(best, __shfl_xor_sync(~0u, best, off));
        const uint32_t who = __ballot_sync(~0u, cost == best);
        int32_t chosen = __shfl_sync(~0u, len, __ffs(who) - 1);
        if (best == INT64_MAX)                           // longer than any of these
            chosen = (int32_t)((members + a.common_budget - 1) / a.common_budget);
        if (tid == 0) {
            run_len[0] = chosen;
            run_len[1] = own;
        }
    }
    __syncthreads();
    const int32_t common = run_len[0], own = run_len[1];

    // ---- the sequences' parts, and how many records there are of each kind
    int32_t carry = 0;
    for (int32_t base = 0; base < a.B; base += kPlanThreads) {
        const int32_t b = base + tid;
        Sequence s{};
        if (b < a.B) s = sequence_at(a, b, false);
        const int32_t n = parts_of(s.prefix_tiles, common, s.dealt) +
                          parts_of(s.own_tiles, own, true);
        const int32_t at = block_prefix(n, carry, scans);
        if (b < a.B) a.part_prefix[b] = at;
    }
    if (tid == 0) a.part_prefix[a.B] = carry;
    int32_t n_common = 0, n_own = 0;
    for (int32_t g = tid; g < groups; g += kPlanThreads) {
        const Group x = group_at(a, g, false);
        if (x.keys > 0)
            n_common += (ceil_div(x.seqs, a.tile_seqs) + 1) / 2 *
                        ceil_div(key_tiles(a, 0, x.keys), common);
    }
    for (int32_t b = tid; b < a.B; b += kPlanThreads)
        n_own += ceil_div(sequence_at(a, b, false).own_tiles, own);
    n_common = (int32_t)block_sum(n_common, sums);
    n_own = (int32_t)block_sum(n_own, sums);
    const bool fits = n_common + n_own <= a.cap_records && carry <= a.cap_parts;
    if (!fits) {                             // cannot be: the lengths above allow for it
        if (tid == 0) pkv::report(a.status, PKV_STATUS_WORKSPACE_OVERFLOW);
        for (int32_t b = tid; b <= a.B; b += kPlanThreads) a.part_prefix[b] = 0;
    }
    if (tid == 0) {
        a.ctrl[0] = fits ? n_common + n_own : 0;
        a.ctrl[1] = 0;
    }
    if (!fits) return;
    // ---- records: the common ones spread over the first three quarters of the own ones, so
    // that the two kinds run side by side and short items come last
    const int32_t spread = max(1, n_own - n_own / 4);
    auto common_at = [&](int32_t i) {
        return n_own == 0 ? i : i + (int32_t)((int64_t)i * spread / n_common);
    };
    auto own_at = [&](int32_t j) {
        const int64_t before = ((int64_t)(j + 1) * n_common + spread - 1) / spread;
        return j + (int32_t)min(before, (int64_t)n_common);
    };
    carry = 0;
    for (int32_t base = 0; base < groups; base += kPlanThreads) {
        const int32_t g = base + tid;
        Group x{};
        int32_t pairs = 0, cuts = 0, tiles = 0;
        if (g < groups) x = group_at(a, g, false);
        if (x.keys > 0) {
            tiles = ceil_div(x.seqs, a.tile_seqs);
            pairs = (tiles + 1) / 2;
            cuts = ceil_div(key_tiles(a, 0, x.keys), common);
        }
        const int32_t at = block_prefix(pairs * cuts, carry, scans);
        for (int32_t i = 0; i < pairs * cuts; ++i) {
            const int32_t cut = i / pairs, pair = i - cut * pairs;
            Record r{};
            r.b0 = x.first + pair * 2 * a.tile_seqs;
            r.seqs = min(2 * a.tile_seqs, x.first + x.seqs - r.b0);
            r.table = a.table[x.first];
            r.key_lo = cut * common * a.tile_keys;
            r.key_hi = min(x.keys, (cut + 1) * common * a.tile_keys);
            r.part = cut * (r.seqs <= a.tile_seqs ? min(2, common) : 1);
            // no member has keys: nobody's table to read
            if (r.table == INT32_MAX) r.key_hi = r.key_lo;
            a.records[common_at(at + i)] = r;
        }
    }
    carry = 0;
    for (int32_t base = 0; base < a.B; base += kPlanThreads) {
        const int32_t b = base + tid;
        Sequence s{};
        if (b < a.B) s = sequence_at(a, b, false);
        const int32_t n = ceil_div(s.own_tiles, own);
        const int32_t at = block_prefix(n, carry, scans);
        const int32_t first = parts_of(s.prefix_tiles, common, s.dealt);
        const int32_t origin = tile_origin(a, s.prefix);
        for (int32_t i = 0; i < n; ++i) {
            Record r{};
            r.b0 = r.table = b;
            r.seqs = 1;
            r.key_lo = i == 0 ? s.prefix : origin + i * own * a.tile_keys;
            r.key_hi = min(s.ctx, origin + (i + 1) * own * a.tile_keys);
            r.part = first + i * min(2, own);
            a.records[own_at(at + i)] = r;
        }
    }
}

// ----------------------------------------------------------------- attention
template <int D>
struct __align__(1024) Smem {
    static constexpr int kTile = kKeys * D * 2;            // bytes of a Q, K or V tile
    static constexpr int kSlots = D == 128 ? 5 : 12;       // K and V tiles in turn
    unsigned char q[2][kTile];
    unsigned char kv[kSlots][kTile];
    uint64_t q_full[2], q_empty[2];
    uint64_t kv_full[kSlots], kv_empty[kSlots];
    uint64_t s_full[2], p_full[2], pv_done[2], o_free[2];
    uint64_t item_full[kItemRing], item_empty[kItemRing];
    uint64_t mma_done;
    uint4 mask[kMaskRing];                                 // keys of a tile that count
    struct Item {
        int32_t b0, seqs, key_lo, key_hi, origin, tiles, kvh, head_tile, part;
        int32_t group;                                     // softmax group of the first tile
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

// The K or V rows of a key tile by cp.async: lane l resolves rows l, l + 32, ...; then
// D / 8 lanes copy a row, each 16-byte chunk to where a 128-byte-swizzled box would put
// it.  Rows that do not count are left as they are.
template <int D>
__device__ __forceinline__ void gather_rows(const int64_t (&src)[4], const __nv_bfloat16* pool,
                                            unsigned char* dst, int lane) {
    constexpr int kChunks = D / 8, kRowsPer = 32 / kChunks;
    const int c = lane % kChunks, sub = lane / kChunks;
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll 4
        for (int i = 0; i < 32 / kRowsPer; ++i) {
            const int rl = i * kRowsPer + sub;
            const int64_t e = __shfl_sync(0xffffffffu, src[g], rl);
            const int r = g * 32 + rl;
            if (e >= 0)
                cp_async16(dst + (c >> 3) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                           pool + e + c * 8, 16);
        }
}

// kGather: rows gathered (block sizes that are no multiple of 8).  kPolls: the waits take
// their limit from the arguments (pkv_set_wait_poll_limit).
template <int D, bool kGather, bool kPolls>
__global__ void __launch_bounds__(kThreads, 1)
    shared_kernel(const __grid_constant__ Maps maps, const SharedArgs a) {
    using S = Smem<D>;
    using Item = typename S::Item;
    constexpr int kTile = S::kTile, kSlots = S::kSlots, kBlocks = D / 64;
    const uint32_t polls = kPolls ? a.wait_polls : (uint32_t)PKV_DEFAULT_WAIT_POLLS;
    extern __shared__ unsigned char smem_raw[];
    S& s = *reinterpret_cast<S*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        s.abort_flag = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 2);
            mbar_init(&s.p_full[i], 4);
            mbar_init(&s.pv_done[i], 1);
            mbar_init(&s.o_free[i], 4);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&s.kv_full[i], 1);
            mbar_init(&s.kv_empty[i], 1);
        }
        for (int i = 0; i < kItemRing; ++i) {
            mbar_init(&s.item_full[i], 1);
            mbar_init(&s.item_empty[i], kItemReaders);
        }
        mbar_init(&s.mma_done, 2);
        mbar_init_fence();
    }
    if (warp == 9) tmem_alloc(&s.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    pkv::wait_for_predecessor();             // the plan's records
    pkv::allow_dependent_launch();           // the combine reads the plan's parts at once
    const int32_t units = a.Hkv * a.head_tiles;
    const int64_t n_items64 = (int64_t)a.ctrl[0] * units;
    const uint32_t n_items = (uint32_t)n_items64;
    uint32_t fills = 0, q_fills = 0;         // the producer's

    // Item I from the producer's ring; false: none in time.
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

    if (warp == 8) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            tma_prefetch_desc(&maps.q);
            tma_prefetch_desc(&maps.q_one);
            if (!kGather) {
                tma_prefetch_desc(&maps.k);
                tma_prefetch_desc(&maps.v);
                tma_prefetch_desc(&maps.k_edge);
                tma_prefetch_desc(&maps.v_edge);
            }
        }
        const uint32_t wrap = n_items + gridDim.x - 1;     // the last draw resets the counter
        auto draw = [&]() {
            return lane == 0 ? atomicInc((unsigned int*)a.ctrl + 1, wrap) : 0u;
        };
        uint32_t tile_no = 0, group = 0;
        bool ok = true, bad_block = false;
        int pend = -1;                       // a gathered slot in flight
        auto land = [&](int slot) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.kv_full[slot]);
        };
        uint32_t next = draw(), it = __shfl_sync(0xffffffffu, next, 0);
        for (uint32_t I = 0; ok; ++I) {
            const int ring = I % kItemRing;
            if (I >= kItemRing && !(ok = warp_wait(&s.item_empty[ring], (I / kItemRing - 1) & 1,
                                                   &s.abort_flag, polls)))
                break;
            if (it >= n_items) {
                if (lane == 0) {
                    s.items[ring].end = 1;
                    mbar_arrive(&s.item_full[ring]);
                }
                break;
            }
            next = draw();                   // needed only behind this item's loads
            const int32_t rec = (int32_t)(it / units), unit = (int32_t)(it - rec * units);
            const int4 r0 = *reinterpret_cast<const int4*>(a.records + rec);
            const int2 r1 = *reinterpret_cast<const int2*>(&a.records[rec].key_hi);
            Item x;
            x.b0 = r0.x;
            x.seqs = r0.y;
            const int32_t* table = a.bt + (int64_t)r0.z * a.MB;
            x.key_lo = r0.w;
            x.key_hi = r1.x;
            x.part = r1.y;
            x.origin = tile_origin(a, x.key_lo);
            x.tiles = x.key_hi > x.key_lo ? ceil_div(x.key_hi - x.origin, a.tile_keys) : 0;
            x.kvh = unit / a.head_tiles;
            x.head_tile = unit - x.kvh * a.head_tiles;
            x.end = 0;
            const bool pair = x.seqs > a.tile_seqs;
            x.group = pair ? 0 : group;
            if (lane == 0) {
                s.items[ring] = x;
                mbar_arrive(&s.item_full[ring]);
            }
            if (x.tiles > 0) {
                // ---- Q: one or two row tiles
                const CUtensorMap* qm = x.seqs == 1 ? &maps.q_one : &maps.q;
                const uint32_t q_bytes =
                    (uint32_t)(kBlocks * 128 * a.tile_heads * (x.seqs == 1 ? 1 : a.tile_seqs));
                for (int t = 0; t < (pair ? 2 : 1); ++t) {
                    const int slot = q_fills & 1;
                    if (q_fills >= 2 &&
                        !(ok = warp_wait(&s.q_empty[slot], (q_fills / 2 - 1) & 1, &s.abort_flag,
                                         polls)))
                        break;
                    if (lane == 0) {
                        mbar_expect_tx(&s.q_full[slot], q_bytes);
                        for (int hf = 0; hf < kBlocks; ++hf)
                            tma_load_4d(s.q[slot] + hf * kHalf, qm, &s.q_full[slot], hf * 64,
                                        x.head_tile * a.tile_heads, x.kvh,
                                        x.b0 + t * a.tile_seqs);
                    }
                    ++q_fills;
                }
                if (!ok) break;
                if (!pair) group ^= x.tiles & 1;
            }
            // ---- K and V tiles
            for (int32_t j = 0; j < x.tiles && ok; ++j, ++tile_no) {
                const int32_t key0 = x.origin + j * a.tile_keys;
                const int32_t lo = max(x.key_lo - key0, 0);
                const int32_t hi = min(x.key_hi - key0, a.tile_keys);
                uint32_t valid[4];
                int64_t src[4];              // kGather: element offsets of rows, -1: none
                int32_t row = -1;            // else: the pool row of this lane's box
                const bool full = lo == 0 && hi == a.tile_keys;
                const int32_t box = full ? a.box : a.edge_box;
                if constexpr (kGather) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int32_t i = g * 32 + lane, key = key0 + i;
                        src[g] = -1;
                        if (i >= lo && i < hi) {
                            const int32_t blk = __ldg(table + key / a.bs);
                            if ((unsigned)blk < (unsigned)a.NB)
                                src[g] = (((int64_t)blk * a.bs + key % a.bs) * a.Hkv + x.kvh) * D;
                            else
                                bad_block = true;
                        }
                        valid[g] = __ballot_sync(0xffffffffu, src[g] >= 0);
                    }
                } else {
                    const int32_t i = lane * box, key = key0 + i;
                    const bool wanted = i < hi && i + box > lo;
                    if (wanted) {
                        const int32_t blk = __ldg(table + key / a.bs);
                        if ((unsigned)blk < (unsigned)a.NB) row = blk * a.bs + key % a.bs;
                        else bad_block = true;
                    }
#pragma unroll
                    for (int w = 0; w < 4; ++w) valid[w] = range_word(lo, hi, w);
                    uint32_t gone = __ballot_sync(0xffffffffu, wanted && row < 0);
                    while (gone) {
                        const int u = __ffs(gone) - 1;
                        gone &= gone - 1;
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            valid[w] &= ~range_word(u * box, (u + 1) * box, w);
                    }
                }
                const int boxes = __popc(__ballot_sync(0xffffffffu, row >= 0));
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++fills) {
                    const int slot = fills % kSlots;
                    if (fills >= kSlots &&
                        !(ok = warp_wait(&s.kv_empty[slot], (fills / kSlots - 1) & 1,
                                         &s.abort_flag, polls)))
                        break;
                    if (kv == 0 && lane == 0)
                        s.mask[tile_no % kMaskRing] =
                            make_uint4(valid[0], valid[1], valid[2], valid[3]);
                    if constexpr (kGather) {
                        gather_rows<D>(src, kv ? a.vc : a.kc, s.kv[slot], lane);
                        asm volatile("cp.async.commit_group;" ::: "memory");
                        if (pend >= 0) {     // the tile before this one has landed
                            asm volatile("cp.async.wait_group 1;" ::: "memory");
                            land(pend);
                        }
                        pend = slot;
                    } else {
                        if (lane == 0) {
                            if (boxes > 0)
                                mbar_expect_tx(&s.kv_full[slot],
                                               (uint32_t)(boxes * box * 128 * kBlocks));
                            else
                                mbar_arrive(&s.kv_full[slot]);
                        }
                        __syncwarp();
                        if (row >= 0) {
                            const CUtensorMap* m = full ? (kv ? &maps.v : &maps.k)
                                                        : (kv ? &maps.v_edge : &maps.k_edge);
                            for (int hf = 0; hf < kBlocks; ++hf)
                                tma_load_3d(s.kv[slot] + hf * kHalf + lane * box * 128, m,
                                            &s.kv_full[slot], hf * 64, x.kvh, row);
                        }
                    }
                }
            }
            if (!ok) break;
            it = __shfl_sync(0xffffffffu, next, 0);
        }
        if (pend >= 0) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            land(pend);
        }
        // every CTA draws until it gets nothing, so that the counter ends where it began
        for (it = __shfl_sync(0xffffffffu, next, 0); it < n_items;)
            it = __shfl_sync(0xffffffffu, draw(), 0);
        if (__any_sync(0xffffffffu, bad_block) && lane == 0)
            pkv::report(a.status, PKV_STATUS_BAD_BLOCK_ID);
        if (!ok && lane == 0) give_up(s, a.status);
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------------------ MMA issuers
        if (lane == 0) {
            const uint32_t id_qk = umma_idesc_bf16(kRows, kKeys, false);
            const uint32_t id_pv = umma_idesc_bf16(kRows, D, true);
            const uint64_t qd0 = umma_desc_sw128(saddr(s.q[0]), 16, 1024);
            const uint64_t kd0 = umma_desc_sw128(saddr(s.kv[0]), 16, 1024);
            const uint64_t vd0 = umma_desc_sw128(saddr(s.kv[0]), kHalf, 1024);
            uint32_t n[2] = {0, 0};          // products of each group so far
            uint32_t o_uses[2] = {0, 0};     // items each group's O was used for
            uint32_t q_uses = 0;             // Q tiles so far
            uint32_t tile_no = 0;
            bool ok = true;
            for (uint32_t I = 0; ok; ++I) {
                Item x;
                if (!(ok = next_item(I, x, false)) || x.end) break;
                if (x.tiles == 0) continue;
                const bool pair = x.seqs > a.tile_seqs;
                if (warp == 9) {
                    for (int t = 0; t < (pair ? 2 : 1) && ok; ++t)
                        ok = mbar_wait(&s.q_full[(q_uses + t) & 1], ((q_uses + t) / 2) & 1,
                                       &s.abort_flag, polls);
                    if (!ok) break;
                    for (int32_t j = 0; j < x.tiles && ok; ++j) {
                        const uint32_t fill = 2 * (tile_no + j), slot = fill % kSlots;
                        if (!(ok = mbar_wait(&s.kv_full[slot], (fill / kSlots) & 1, &s.abort_flag,
                                             polls)))
                            break;
                        const uint64_t kd = kd0 + (uint64_t)(slot * (kTile >> 4));
                        for (int t = 0; t < (pair ? 2 : 1); ++t) {
                            const int g = pair ? t : (x.group + j) & 1;
                            // this S still holds the group's last P until its product is done
                            if (n[g] > 0 && !(ok = mbar_wait(&s.pv_done[g], (n[g] - 1) & 1,
                                                             &s.abort_flag, polls)))
                                break;
                            tc_fence_after();
                            const uint64_t qd =
                                qd0 + (uint64_t)(((q_uses + t) & 1) * (kTile >> 4));
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk) {
                                const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                                umma_bf16(tmem + g * kKeys, qd + off, kd + off, id_qk, kk > 0);
                            }
                            umma_commit(&s.s_full[g]);
                            mbar_arrive(&s.s_full[g]);     // passes on the producer's mask
                            ++n[g];
                        }
                        if (!ok) break;
                        umma_commit(&s.kv_empty[slot]);
                    }
                    if (!ok) break;
                    for (int t = 0; t < (pair ? 2 : 1); ++t)
                        umma_commit(&s.q_empty[(q_uses + t) & 1]);
                    q_uses += pair ? 2 : 1;
                } else {
                    for (int32_t j = 0; j < x.tiles && ok; ++j) {
                        const uint32_t fill = 2 * (tile_no + j) + 1, slot = fill % kSlots;
                        const uint64_t vd = vd0 + (uint64_t)(slot * (kTile >> 4));
                        const int steps =
                            (min(x.key_hi - x.origin - j * a.tile_keys, a.tile_keys) + 15) / 16;
                        for (int t = 0; t < (pair ? 2 : 1); ++t) {
                            const int g = pair ? t : (x.group + j) & 1;
                            const bool first = pair ? j == 0 : j < 2;
                            if (!(ok = mbar_wait(&s.p_full[g], n[g] & 1, &s.abort_flag, polls)))
                                break;
                            if (first) {
                                if (o_uses[g] > 0 &&
                                    !(ok = mbar_wait(&s.o_free[g], (o_uses[g] - 1) & 1,
                                                     &s.abort_flag, polls)))
                                    break;
                                ++o_uses[g];
                            }
                            if (!(ok = mbar_wait(&s.kv_full[slot], (fill / kSlots) & 1,
                                                 &s.abort_flag, polls)))
                                break;
                            tc_fence_after();
                            for (int kk = 0; kk < steps; ++kk)
                                umma_bf16_tmem_a(tmem + 256 + g * 128, tmem + g * kKeys + kk * 8,
                                                 vd + (kk * 2048 >> 4), id_pv,
                                                 kk > 0 || !first ? 1u : 0u);
                            umma_commit(&s.pv_done[g]);
                            ++n[g];
                        }
                        if (!ok) break;
                        umma_commit(&s.kv_empty[slot]);
                    }
                }
                tile_no += x.tiles;
            }
            if (!ok) give_up(s, a.status);
            // every product of both issuers has finished before TMEM is freed
            umma_commit(&s.mma_done);
            mbar_drain(&s.mma_done, 0);
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ softmax
        const int g = warp >> 2, i = tid & 127;            // group; row = TMEM lane
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_col = tmem + lanes + g * kKeys, o_col = tmem + lanes + 256 + g * 128;
        const int32_t my_seq = i / a.tile_heads, my_head = i - my_seq * a.tile_heads;
        uint32_t n = 0, tile_no = 0;         // this group's products; the CTA's tiles
        bool ok = true;
        for (uint32_t I = 0; ok; ++I) {
            Item x;
            if (!(ok = next_item(I, x, true)) || x.end) break;
            const bool pair = x.seqs > a.tile_seqs;
            const int32_t j0 = pair ? 0 : (x.group == g ? 0 : 1), step = pair ? 1 : 2;
            if (j0 >= x.tiles) {
                tile_no += x.tiles;
                continue;
            }
            const int32_t seqs = pair ? (g == 0 ? a.tile_seqs : x.seqs - a.tile_seqs) : x.seqs;
            const int32_t head = x.head_tile * a.tile_heads + my_head;
            const bool mine = my_seq < seqs && my_seq < a.tile_seqs && head < a.G;
            const bool active = (warp & 3) * 32 < min(seqs, a.tile_seqs) * a.tile_heads;
            float m_run = -INFINITY, l_run = 0.f;
            for (int32_t j = j0; j < x.tiles; j += step, ++n) {
                const uint32_t t = tile_no + j;
                if (!(ok = warp_wait(&s.s_full[g], n & 1, &s.abort_flag, polls))) break;
                tc_fence_after();
                const uint4 mk = s.mask[t % kMaskRing];
                const uint32_t mask[4] = {mk.x, mk.y, mk.z, mk.w};
                const bool whole = (mk.x & mk.y & mk.z & mk.w) == ~0u;
                if (active) {
                    uint32_t pw[64];
                    float sum = 0.f;
                    // P against `neg_m`, 32 columns at a time, and its sum
                    auto exp_pass = [&](float neg_m) {
                        const uint64_t scale2 = pk2(a.scale_log2, a.scale_log2);
                        const uint64_t neg2 = pk2(neg_m, neg_m);
                        uint64_t l2[2] = {0, 0};
#pragma unroll
                        for (int cc = 0; cc < 4; ++cc) {
                            float sv[32];
                            tmem_ld32(s_col + cc * 32, sv);
                            tmem_wait_ld();
                            if (!whole) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    sv[e] = (mask[cc] >> e) & 1 ? sv[e] : -INFINITY;
                            }
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float x0, x1;
                                up2(fma2(pk2(sv[2 * e], sv[2 * e + 1]), scale2, neg2), x0, x1);
                                const float p0 = pkv::fast_exp2(x0), p1 = pkv::fast_exp2(x1);
                                l2[e & 1] = add2(l2[e & 1], pk2(p0, p1));
                                pw[cc * 16 + e] = pkv::pack_bf16(p0, p1);
                            }
                        }
                        float s0, s1, s2, s3;
                        up2(l2[0], s0, s1);
                        up2(l2[1], s2, s3);
                        sum = (s0 + s1) + (s2 + s3);
                    };
                    bool redo = j == j0;
                    if (!redo) {
                        exp_pass(-m_run);
                        redo = __any_sync(0xffffffffu, mine && !(sum <= kSumTrigger));
                    }
                    if (redo) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int cc = 0; cc < 4; ++cc) {
                            float sv[32];
                            tmem_ld32(s_col + cc * 32, sv);
                            tmem_wait_ld();
                            if (!whole) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    sv[e] = (mask[cc] >> e) & 1 ? sv[e] : -INFINITY;
                            }
                            float part[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) part[e] = fmaxf(sv[e], sv[4 + e]);
#pragma unroll
                            for (int c = 8; c < 32; c += 8)
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    part[e] = max3(part[e], sv[c + e], sv[c + 4 + e]);
                            mx = max3(mx, fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
                        }
                        mx *= a.scale_log2;                // scale > 0 keeps the order
                        const bool raise = mine && mx > m_run + kRescaleThreshold;
                        float alpha = 1.f;
                        if (raise) {
                            alpha = m_run == -INFINITY ? 0.f : pkv::fast_exp2(m_run - mx);
                            m_run = mx;
                            l_run *= alpha;
                        }
                        // this S was computed behind the group's last P V: O is at rest
                        if (j > j0 && __any_sync(0xffffffffu, raise)) {
#pragma unroll
                            for (int cc = 0; cc < D / 32; ++cc) {
                                float ov[32];
                                tmem_ld32(o_col + cc * 32, ov);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) ov[e] *= alpha;
                                tmem_st32(o_col + cc * 32, ov);
                            }
                        }
                        exp_pass(m_run == -INFINITY ? 0.f : -m_run);
                    }
                    l_run += sum;
                    // P over the first 64 columns of S
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        float pf[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) pf[e] = __uint_as_float(pw[half * 32 + e]);
                        tmem_st32(s_col + half * 32, pf);
                    }
                    tmem_wait_st();
                }
                if (!whole && (!pair || g == 0)) {
                    // V rows of keys that do not count may hold anything: thread i clears
                    // row i (both groups of a pair use the same tile, the first clears it)
                    const uint32_t fill = 2 * t + 1, slot = fill % kSlots;
                    if (!(ok = warp_wait(&s.kv_full[slot], (fill / kSlots) & 1, &s.abort_flag,
                                         polls)))
                        break;
                    if (!((mask[warp & 3] >> lane) & 1)) {
#pragma unroll
                        for (int hf = 0; hf < kBlocks; ++hf)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                *reinterpret_cast<uint4*>(s.kv[slot] + hf * kHalf + i * 128 +
                                                          c * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.p_full[g]);
            }
            if (!ok) break;
            tile_no += x.tiles;
            // ---- this group's part, or the result where there is no other
            if (!(ok = warp_wait(&s.pv_done[g], (n - 1) & 1, &s.abort_flag, polls))) break;
            tc_fence_after();
            if (active) {
                const int32_t b = x.b0 + (pair && g == 1 ? a.tile_seqs : 0) + my_seq;
                int32_t first = 0, parts = 0;
                if (mine) {
                    first = a.part_prefix[b];
                    parts = a.part_prefix[b + 1] - first;  // 0: a sequence without keys
                }
                const int64_t row = x.kvh * a.G + head;
                const int64_t at = ((int64_t)first + x.part + j0) * a.Hq + row;
                const bool some = l_run > 0.f || l_run != l_run;
                const float inv = some ? 1.f / l_run : 0.f;
                const bool wide = ((uintptr_t)a.out & 31) == 0;
                __nv_bfloat16* out = a.out + ((int64_t)b * a.Hq + row) * D;
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                    float ov[32];
                    tmem_ld32(o_col + cc * 32, ov);
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
                if (parts > 1) a.part_ml[at] = make_float2(0.5f * m_run, l_run);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.o_free[g]);
        }
        if (!ok && lane == 0) give_up(s, a.status);
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (s.abort_flag && warp == 8 && lane == 0) {
        // some role gave up: every copy issued lands before the CTA exits
        for (uint32_t back = 1; back <= (uint32_t)kSlots && back <= fills; ++back) {
            const uint32_t f = fills - back;
            mbar_drain(&s.kv_full[f % kSlots], (f / kSlots) & 1);
        }
        for (uint32_t back = 1; back <= 2 && back <= q_fills; ++back) {
            const uint32_t f = q_fills - back;
            mbar_drain(&s.q_full[f & 1], (f / 2) & 1);
        }
    }
    if (warp == 9) tmem_dealloc(tmem, 512);
}

// ----------------------------------------------------------------------- host
struct Layout {
    int32_t box, edge_box, tile_keys, tile_heads, head_tiles, tile_seqs;
    int32_t cap_records, cap_parts, common_budget;
    size_t off_prefix, off_group, off_table, off_records, off_ml, off_o, total;
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
    // Parts.  A run of tiles has two at most.  Own runs are long enough for 16 kSms items in
    // all, and one more for each sequence; common runs, so long that their items could be
    // 4 kSms of 2 tile_seqs sequences each, and one more for each sequence.  Neither is more
    // than the tiles there can be.
    const int64_t units = (int64_t)c.num_kv_heads * L.head_tiles;
    const int64_t tiles = (int64_t)batch * (ceil_div(max_ctx, L.tile_keys) + 1);
    const int64_t own = (16 * kSms + units - 1) / units;
    const int64_t common = (2 * (int64_t)L.tile_seqs * 4 * kSms + units - 1) / units;
    L.common_budget = (int32_t)(common < tiles ? common : tiles);
    if (L.common_budget < 1) L.common_budget = 1;
    const int64_t parts = 2 * (L.common_budget + (own < tiles ? own : tiles) + 2 * (int64_t)batch + 2);
    if (parts > (1 << 30) || parts * units > (1LL << 31)) return false;
    L.cap_parts = L.cap_records = (int32_t)parts;
    auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
    L.off_prefix = 256;
    L.off_group = align(L.off_prefix + sizeof(int32_t) * ((size_t)batch + 1));
    L.off_table = align(L.off_group + sizeof(int32_t) * (size_t)batch);
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
    if (!workspace) return PKV_ERR_NULL_POINTER;
    if ((uintptr_t)workspace & 15) return PKV_ERR_MISALIGNED;
    Layout L;
    if (!layout(batch, num_q_heads, max_context_len, cache, L)) return PKV_ERR_UNSUPPORTED;
    if (workspace_bytes < L.total) return PKV_ERR_WORKSPACE_TOO_SMALL;
    char* ws = (char*)(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    a = SharedArgs{};
    a.ctrl = (int32_t*)ws;
    a.part_prefix = (int32_t*)(ws + L.off_prefix);
    a.group = (int32_t*)(ws + L.off_group);
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
    a.tile_heads = L.tile_heads;
    a.head_tiles = L.head_tiles;
    a.tile_seqs = L.tile_seqs;
    a.cap_records = L.cap_records;
    a.cap_parts = L.cap_parts;
    a.common_budget = L.common_budget;
    a.status = status;
    a.wait_polls = pkv_wait_polls();
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
    return PKV_OK;
}

int launch_plan(const SharedArgs& a, cudaStream_t s) {
    plan_kernel<<<1, kPlanThreads, 0, s>>>(a);
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
