// paged_prefill_varlen_fp8: causal varlen prefill over chunks whose cached
// prefix lies in an e4m3 cache (scales per cache block and kv head).
//
// What it computes: as paged_prefill_varlen, with the prefix rows code * scale.
//
// Design.  Prefill of long chunks is bound by the tensor pipe, and a prefix row is read
// once per 128-query tile and q head, so turning codes into operands inside the
// attention kernel would repeat the conversion tens to hundreds of times
// beside the softmax, the busiest role there.  (For one to three tiles a sequence it
// would not; those calls pay for the pass: 12 us of 37 for 3 chunks of 20..301 queries.)
// Instead one pass writes the
// prefix rows once as bf16 into the workspace, as cache blocks of 128 rows,
// and the bf16 kernel attends over them: it takes its fastest path (whole-tile
// TMA boxes) whatever the e4m3 cache's own block size.  With a power-of-two
// scale, as kv_store_fp8 writes, the bf16 row is exact; the weights are rounded to bf16
// for the product with V, as that kernel does.  The pass moves 3 bytes
// per prefix entry (1 read, 2 written), most of which the attention then finds
// in L2.  Batches whose prefixes would exceed kExpandBytes run in groups of
// sequences, one after another over the same workspace.
//
// A chunk of few queries on a long prefix has few (q tile, head) work items, each
// a serial walk over its key tiles.  Where they could not fill the GPU, a tile's
// keys are split into work items of their own, whose partial results a combine
// kernel merges (3 chunks of 20..301 queries on 500..6000 cached keys, 16 heads:
// 40 us for the attention without splits, 19 with them).
#include "fp8_common.cuh"
#include "prefill_common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kChunkRows = 16;               // prefix rows per CTA
constexpr int kBatch = 4;                    // vectors a lane has in flight
constexpr int kBlock = 128;                  // rows per workspace cache block
constexpr int64_t kExpandBytes = 4100000000; // K and V rows of a group, where >= 1 fits

struct ExpandArgs {
    const uint8_t* kc;
    const uint8_t* vc;
    const float* ks;
    const float* vs;
    const int32_t* bt;
    __nv_bfloat16* ko;                       // [sequences * rows_per_seq, Hkv, D]
    __nv_bfloat16* vo;
    int32_t* table;                          // [sequences, rows_per_seq / kBlock]
    int32_t MB, NB, bs, Hkv, D, rows_per_seq;
    int32_t vec_shift;                       // log2 of the vectors of a row, -1: not a power of two
};

__device__ __forceinline__ uint32_t to_bf16x2(uint32_t f16x2, float s) {
    const float2 f = pkv::f16x2_to_float2(f16x2);
    return pkv::pack_bf16(f.x * s, f.y * s);
}

// 32 bytes to global memory in one instruction (address 32-byte aligned).
__device__ __forceinline__ void st_global_32b(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// CTA (x, y): prefix rows 16x .. 16x + 15 of sequence y.  A row that cannot be
// read (block id or scale out of range) is written as zeros and reported.
__global__ void __launch_bounds__(kThreads) expand_prefix_kernel(ExpandArgs e,
                                                                 pkv::PrefillArgs p) {
    pkv::allow_dependent_launch();
    const int32_t b = blockIdx.y, r0 = blockIdx.x * kChunkRows;
    if (r0 % kBlock == 0 && threadIdx.x == 0)
        e.table[(int64_t)b * (e.rows_per_seq / kBlock) + r0 / kBlock] =
            (int32_t)(((int64_t)b * e.rows_per_seq + r0) / kBlock);
    int32_t q0, lq, lk;
    if (!pkv::seq_lengths(p, b, q0, lq, lk, false)) return;   // the plan kernel reports it
    const int32_t rows = min(lk - lq - r0, kChunkRows);
    if (rows <= 0) return;
    const int32_t vecs = e.Hkv * (e.D / 16);                  // 16-code vectors per row
    const int32_t half = rows * vecs;                         // K's vectors, then V's
    const int head_shift = e.D == 128 ? 3 : 2;                // vectors of a head, log2
    // a chunk of 16 rows lies in one cache block where the block size allows
    const bool one_block = e.bs % kChunkRows == 0;
    const int32_t blk0 = one_block ? __ldg(e.bt + (int64_t)b * e.MB + r0 / e.bs) : 0;
    const int32_t off0 = r0 % e.bs;
    uint32_t bad = 0;
    // kBatch vectors a lane at once: a vector is three loads, of which the scale's
    // and the codes' addresses need the block id
    for (int32_t i0 = threadIdx.x; i0 < 2 * half; i0 += kBatch * kThreads) {
        int32_t blk[kBatch], row[kBatch], col[kBatch];       // row of the chunk; vector of the row
        float s[kBatch];
        uint4 w[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int32_t i = i0 + u * kThreads;
            const int32_t j = i < half ? i : i - half;
            row[u] = e.vec_shift >= 0 ? j >> e.vec_shift : j / vecs;
            col[u] = j - row[u] * vecs;
            blk[u] = i >= 2 * half ? -1
                     : one_block   ? blk0
                                   : __ldg(e.bt + (int64_t)b * e.MB + (r0 + row[u]) / e.bs);
            if (i < 2 * half && (unsigned)blk[u] >= (unsigned)e.NB) {
                bad |= PKV_STATUS_BAD_BLOCK_ID;
                blk[u] = -1;
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const bool is_v = i0 + u * kThreads >= half;
            s[u] = 0.f;
            w[u] = make_uint4(0, 0, 0, 0);
            if (blk[u] < 0) continue;
            s[u] = __ldg((is_v ? e.vs : e.ks) + (int64_t)blk[u] * e.Hkv + (col[u] >> head_shift));
            w[u] = pkv::ld_stream16((is_v ? e.vc : e.kc) +
                                    (((int64_t)blk[u] * e.bs +
                                      (one_block ? off0 + row[u] : (r0 + row[u]) % e.bs)) * vecs +
                                     col[u]) * 16);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int32_t i = i0 + u * kThreads;
            if (i >= 2 * half) continue;
            float sc = s[u];
            if (!pkv::scale_ok(sc)) {
                if (blk[u] >= 0) bad |= PKV_STATUS_BAD_SCALE;
                sc = 0.f;
                w[u] = make_uint4(0, 0, 0, 0);
            }
            uint32_t h[8];
            pkv::e4m3x4_to_f16x4(w[u].x, h[0], h[1]);
            pkv::e4m3x4_to_f16x4(w[u].y, h[2], h[3]);
            pkv::e4m3x4_to_f16x4(w[u].z, h[4], h[5]);
            pkv::e4m3x4_to_f16x4(w[u].w, h[6], h[7]);
#pragma unroll
            for (int x = 0; x < 8; ++x) h[x] = to_bf16x2(h[x], sc);
            st_global_32b((i >= half ? e.vo : e.ko) +
                              (((int64_t)b * e.rows_per_seq + r0 + row[u]) * vecs + col[u]) * 16,
                          h);
        }
    }
    if (bad) pkv::report(p.status, bad);
}

// CTA r: query row r, a warp a head at a time: merges the row's splits.  Rows of
// unsplit tiles are the attention kernel's.
constexpr int kCombineWarps = 8;

template <int D>
__global__ void __launch_bounds__(kCombineWarps * 32) combine_splits_kernel(pkv::PrefillArgs p) {
    constexpr int E = D / 32;
    __shared__ int32_t owner;                // sequence whose row this is
    const int32_t r = blockIdx.x;
    if (threadIdx.x == 0) owner = -1;
    __syncthreads();
    int32_t q0, lq, lk;
    for (int32_t b = threadIdx.x; b < p.B; b += kCombineWarps * 32)
        if (pkv::seq_lengths(p, b, q0, lq, lk, false) && r >= q0 && r < q0 + lq) owner = b;
    __syncthreads();
    // the attention kernel's partial results; every CTA waits, so that this grid
    // never ends before that one
    pkv::wait_for_predecessor();
    if (owner < 0) return;
    pkv::seq_lengths(p, owner, q0, lq, lk, false);
    const int32_t n = pkv::key_splits(p, pkv::key_tiles(lk - lq, (r - q0) / pkv::kPrefillTileQ));
    if (n == 1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int32_t h = warp; h < p.Hq; h += kCombineWarps) {
        const int64_t at = (int64_t)r * p.Hq + h, step = (int64_t)p.total_q * p.Hq;
        float M = -INFINITY;
#pragma unroll 4
        for (int32_t s = 0; s < n; ++s) M = fmaxf(M, p.part_ml[at + s * step].x);
        const float use = M == -INFINITY ? 0.f : M;
        float L = 0.f, O[E];
#pragma unroll
        for (int e = 0; e < E; ++e) O[e] = 0.f;
#pragma unroll 4
        for (int32_t s = 0; s < n; ++s) {
            const float2 ml = p.part_ml[at + s * step];
            const float f = pkv::fast_exp2(ml.x - use);
            L = fmaf(ml.y, f, L);
            const float* o = p.part_o + (at + s * step) * D + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = *reinterpret_cast<const float2*>(o + e);
                O[e] = fmaf(v.x, f, O[e]);
                O[e + 1] = fmaf(v.y, f, O[e + 1]);
            }
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;           // as for unsplit rows
#pragma unroll
        for (int e = 0; e < E; e += 2)
            *reinterpret_cast<uint32_t*>(p.out + at * D + lane * E + e) =
                pkv::pack_bf16(O[e] * inv, O[e + 1] * inv);
    }
}

template <int D>
int launch_combine(const pkv::PrefillArgs& p, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.total_q, 1, 1);
    cfg.blockDim = dim3(kCombineWarps * 32, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, combine_splits_kernel<D>, p) == cudaSuccess ? PKV_OK
                                                                                : PKV_ERR_CUDA;
}

struct Fp8PrefillLayout {
    int64_t rows_per_seq;
    int32_t group;                           // sequences attended at once
    int32_t split_tiles, max_tiles;          // key tiles of a split (0: none); list entries
    size_t off_table, off_tiles, off_ml, off_o, off_k, off_v, total;
};

// Of a GB300; not asked of the device, because the workspace's size follows from it and
// is a function of the call's sizes alone.
constexpr int kSms = 152;

// Key tiles of a split, 0 for none: as many splits of a tile's keys as bring the
// (q tile, head) items, at most `items`, to two an SM, but none under 16 tiles: a
// split's start and end, its partial rows and the combine cost about as much as
// eight (measured, us, unsplit and at 4, 8, 14, 20 tiles: 64 queries of 32 heads on
// 8000 cached keys 58, 54, 41, 40, 36; 200 on 2000 25, 33, 28, 28, 26; two chunks of
// 100 on 1000 18, 25, 25, 20, 20).
int32_t choose_split(int64_t items, int64_t key_tiles) {
    if (items <= 0) return 0;
    int64_t splits = (2 * kSms + items - 1) / items;
    if (splits > key_tiles / 16) splits = key_tiles / 16;
    return splits < 2 ? 0 : (int32_t)((key_tiles + splits - 1) / splits);
}

Fp8PrefillLayout fp8_prefill_layout(int32_t batch, int32_t total_q, int32_t num_q_heads,
                                    int32_t max_seqlen_k, const pkv_cache_desc& c) {
    Fp8PrefillLayout L{};
    auto align = [](size_t x) { return (x + 255) & ~(size_t)255; };
    L.rows_per_seq = ((int64_t)max_seqlen_k + kBlock) / kBlock * kBlock;
    const int64_t row = (int64_t)c.num_kv_heads * c.head_dim;
    if ((double)L.rows_per_seq * row * 4 > 0x1p60) {         // more than any memory
        L.total = SIZE_MAX;
        return L;
    }
    const int64_t seq_bytes = L.rows_per_seq * row * 4;      // K and V as bf16
    int64_t group = kExpandBytes / seq_bytes;
    if (group > batch) group = batch;
    if (group > 65535) group = 65535;        // the expanding grid's y extent
    if (group < 1) group = 1;
    L.group = (int32_t)group;
    L.off_table = align(pkv_prefill_layout(batch, total_q).total);
    // The sizes reserved below grow with every argument, so that a workspace for the
    // largest call holds the smaller ones; the group and the splits do not.
    int64_t kv_bytes = kExpandBytes > seq_bytes ? kExpandBytes : seq_bytes;
    if (kv_bytes / seq_bytes >= batch) kv_bytes = batch * seq_bytes;
    const int64_t table = kv_bytes / (row * 4 * kBlock) + 1;
    L.off_tiles = align(L.off_table + sizeof(int32_t) * (size_t)table);
    // a sequence's cached and own keys together are max_seqlen_k at most, each part
    // rounded up to tiles
    const int64_t tiles = pkv_prefill_layout(batch, total_q).max_tiles;
    const int64_t key_tiles = L.rows_per_seq / kBlock + 1;
    L.split_tiles = choose_split(tiles * num_q_heads, key_tiles);
    const int64_t splits = L.split_tiles > 0 ? (key_tiles + L.split_tiles - 1) / L.split_tiles : 0;
    L.max_tiles = (int32_t)(tiles * splits);
    // splits * items < 2 * kSms + items where there are any, and items < 2 * kSms
    int64_t items = tiles * num_q_heads;
    if (items > 2 * kSms) items = 2 * kSms;
    int64_t rows = kBlock * (2 * kSms + items);
    const double most = (double)(key_tiles / 16) * num_q_heads * total_q;
    if (most < (double)rows) rows = (int64_t)most;
    if (key_tiles < 32) rows = 0;
    L.off_ml = align(L.off_tiles + sizeof(int2) * 4 * kSms);
    L.off_o = align(L.off_ml + sizeof(float2) * (size_t)rows);
    L.off_k = align(L.off_o + sizeof(float) * (size_t)rows * c.head_dim);
    L.off_v = align(L.off_k + (size_t)(kv_bytes / 2));
    // 256 bytes more: the workspace is 16-byte aligned, the rows are written by 32
    L.total = align(L.off_v + (size_t)(kv_bytes / 2)) + 256;
    return L;
}

struct ExpandCall {
    ExpandArgs e;
    pkv::PrefillArgs p;
    int32_t sequences;
    cudaStream_t s;
};

int enqueue_expand(void* ctx, bool* launched) {
    const ExpandCall& c = *(const ExpandCall*)ctx;
    const dim3 grid((unsigned)(c.e.rows_per_seq / kChunkRows), (unsigned)c.sequences);
    expand_prefix_kernel<<<grid, kThreads, 0, c.s>>>(c.e, c.p);
    *launched = true;
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

extern "C" size_t pkv_paged_prefill_fp8_workspace_bytes(int32_t batch, int32_t total_q,
                                                        int32_t num_q_heads,
                                                        int32_t max_seqlen_k,
                                                        pkv_cache_desc cache) {
    if (batch < 0 || total_q < 0 || num_q_heads <= 0 || max_seqlen_k < 0 ||
        cache.num_kv_heads <= 0 || cache.head_dim <= 0)
        return 0;
    return fp8_prefill_layout(batch, total_q, num_q_heads, max_seqlen_k, cache).total;
}

extern "C" int pkv_paged_prefill_varlen_fp8(
        const void* q, const void* k, const void* v, const void* k_cache, const void* v_cache,
        const float* k_scale, const float* v_scale, const int32_t* cu_seqlens_q,
        const int32_t* cu_seqlens_k, int32_t batch, int32_t total_q, int32_t max_seqlen_q,
        int32_t max_seqlen_k, int32_t num_q_heads, const int32_t* block_tables,
        int32_t max_blocks_per_seq, float scale, void* out, void* workspace,
        size_t workspace_bytes, pkv_cache_desc cache, uint32_t* status, void* stream) {
    // the bf16 prefill's checks, with this call's cache and tables
    pkv::PrefillArgs a{};
    int rc = pkv_prefill_make_args(q, k, v, k_cache, v_cache, cu_seqlens_q, cu_seqlens_k, batch,
                                   total_q, max_seqlen_q, max_seqlen_k, num_q_heads,
                                   block_tables, max_blocks_per_seq, scale, out, workspace,
                                   workspace_bytes, cache, status, a);
    if (rc != PKV_OK || batch == 0 || total_q == 0) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (!block_tables) return pkv_prefill_launch(a, cache.head_dim, s, nullptr);
    if (!k_scale || !v_scale) return PKV_ERR_NULL_POINTER;
    if (((uintptr_t)k_scale | (uintptr_t)v_scale) & 3) return PKV_ERR_MISALIGNED;
    if (cache.block_size > pkv::kFp8MaxBlockSize) return PKV_ERR_BAD_DIMENSION;
    if ((int64_t)cache.num_blocks * cache.block_size >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;
    const Fp8PrefillLayout L =
        fp8_prefill_layout(batch, total_q, num_q_heads, max_seqlen_k, cache);
    if (workspace_bytes < L.total) return PKV_ERR_WORKSPACE_TOO_SMALL;
    if (L.group * L.rows_per_seq >= (1LL << 31)) return PKV_ERR_UNSUPPORTED;
    char* ws = (char*)(((uintptr_t)workspace + 255) & ~(uintptr_t)255);
    ExpandCall c{};
    c.s = s;
    c.e.kc = (const uint8_t*)k_cache;
    c.e.vc = (const uint8_t*)v_cache;
    c.e.ks = k_scale;
    c.e.vs = v_scale;
    c.e.ko = (__nv_bfloat16*)(ws + L.off_k);
    c.e.vo = (__nv_bfloat16*)(ws + L.off_v);
    c.e.table = (int32_t*)(ws + L.off_table);
    c.e.MB = max_blocks_per_seq;
    c.e.NB = cache.num_blocks;
    c.e.bs = cache.block_size;
    c.e.Hkv = cache.num_kv_heads;
    c.e.D = cache.head_dim;
    c.e.rows_per_seq = (int32_t)L.rows_per_seq;
    const int32_t vecs = cache.num_kv_heads * (cache.head_dim / 16);
    c.e.vec_shift = (vecs & (vecs - 1)) == 0 ? __builtin_ctz((unsigned)vecs) : -1;
    const int64_t table_keys = (int64_t)max_blocks_per_seq * cache.block_size;
    a.kc = c.e.ko;
    a.vc = c.e.vo;
    a.bt = c.e.table;
    a.MB = (int32_t)(L.rows_per_seq / kBlock);
    a.bs = kBlock;
    a.max_cached = table_keys < INT32_MAX ? (int32_t)table_keys : INT32_MAX;
    a.skip_long = 1;                         // the workspace has no room for such a sequence
    if (L.split_tiles > 0) {
        a.split_tiles = L.split_tiles;
        a.tiles = (int2*)(ws + L.off_tiles);
        a.max_tiles = L.max_tiles;
        a.part_ml = (float2*)(ws + L.off_ml);
        a.part_o = (float*)(ws + L.off_o);
    }
    const PrefillPrologue pre{enqueue_expand, &c};
    for (int32_t b0 = 0; b0 < batch; b0 += L.group) {
        c.sequences = batch - b0 < L.group ? batch - b0 : L.group;
        c.e.bt = block_tables + (int64_t)b0 * max_blocks_per_seq;
        pkv::PrefillArgs sub = a;
        sub.cu_q = cu_seqlens_q + b0;
        sub.cu_k = cu_seqlens_k + b0;
        sub.B = c.sequences;
        sub.NB = (int32_t)(c.sequences * (L.rows_per_seq / kBlock));
        c.p = sub;
        rc = pkv_prefill_launch(sub, cache.head_dim, s, &pre);
        if (rc == PKV_OK && L.split_tiles > 0)
            rc = cache.head_dim == 128 ? launch_combine<128>(sub, s) : launch_combine<64>(sub, s);
        if (rc != PKV_OK) return rc;
    }
    return PKV_OK;
}
