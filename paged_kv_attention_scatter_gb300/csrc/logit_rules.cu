// apply_logit_rules: penalties for repeated tokens, biases and an allowed-token
// mask on a step's logits, ahead of the sampler.
//
// For entry i of row b, x = logits[b, i] in fp32, n = occurrences of i among
// the row's generated tokens, seen = i occurs in its prompt or generated tokens:
//   seen:  x = x > 0 ? x / r : x * r           (repetition)
//   x -= f * n + p * (n > 0)                    (frequency, presence)
//   x += the row's last bias for token i        (biases)
//   not allowed: x = -inf                       (mask)
//
// Design.  One pass over the logits: a CTA owns a segment of one row's
// vocabulary and keeps a word per entry in shared memory (a bit for the prompt, a
// count for the generated tokens), fills it from the row's whole token list with
// shared-memory atomics (integers, so their order does not matter), then streams
// its segment, 16 bytes a lane where the rows allow.  Those rows' logits are on
// their way to shared memory meanwhile, and words are 16 bits wide where no row
// can have more than 32767 tokens, so that four CTAs fit on a SM: the history's
// round trips and barriers are what a CTA waits for (512 rows of 151936 fp32
// logits with 16..4096 tokens: 125 us with the logits in registers and 32-bit
// words, three CTAs a SM).  The list is read once per segment, out of
// L2, instead of a global table of counts being cleared, filled and read
// (12 bytes a vocabulary entry).  Few entries have a bias, so biases are added
// afterwards to the segment's written entries; the last entry for a token
// is found with an integer maximum in the shared memory that is free by then.
// Rows that do not start on 16 bytes (an odd vocabulary, a stride of their own) are
// staged and written 16 bytes a lane as well, off the boundary in shared memory: 512
// rows of 151937 fp32 logits take 120 us, loaded and written entry by entry 252.
// In place (fp32, out == logits) a vector that no rule changes is not written.
// Bound by memory: the logits in, fp32 out, a mask bit an entry; 106 us, 6.0 TB/s,
// for the rows above, and 91, 6.9 TB/s, without penalties.  Segments of 4096 entries
// measured 110-119 us, 6144 106, 12288 109, 16384 107; 384 or 512 threads 106-113.
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSegment = 8192;            // entries per CTA
constexpr int kSlack = 16;                   // entries more in shared memory, see in_at, out_at
constexpr int kCtas = 4;                     // an SM, 48 KB of fp32 logits and words each
// A word: bit 0 says that a prompt token was this entry, the bits above count
// the generated ones; the entry was seen if the word is not zero.
constexpr uint32_t kInPrompt = 1, kGenerated = 2;

struct RuleArgs {
    const void* logits;
    int64_t stride;                          // entries between rows of logits
    float* out;
    int32_t batch, vocab, segment;
    pkv_logit_rules r;
    uint32_t* status;
    bool in_place;
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

struct RowRules {
    float rep, inv_rep, freq, pres;          // inv_rep = 1 / rep, rounded
    bool penalties;
};

// The words of four entries from `i` on, a multiple of four.
__device__ __forceinline__ uint4 four_words(const uint32_t* words, int i) {
    return reinterpret_cast<const uint4*>(words)[i >> 2];
}
__device__ __forceinline__ uint4 four_words(const uint16_t* words, int i) {
    const uint2 w = reinterpret_cast<const uint2*>(words)[i >> 2];
    return make_uint4(w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16);
}
// Shared-memory atomics are 32 bits wide; 16-bit words do not carry into each other.
__device__ __forceinline__ void count_token(uint32_t* words, uint32_t i, bool prompt) {
    if (prompt) atomicOr(&words[i], kInPrompt);
    else atomicAdd(&words[i], kGenerated);
}
__device__ __forceinline__ void count_token(uint16_t* words, uint32_t i, bool prompt) {
    uint32_t* pair = reinterpret_cast<uint32_t*>(words) + (i >> 1);
    const uint32_t shift = (i & 1) * 16;
    if (prompt) atomicOr(pair, kInPrompt << shift);
    else atomicAdd(pair, kGenerated << shift);
}

__device__ __forceinline__ void cp_async16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(to)),
                 "l"(from)
                 : "memory");
}

__device__ __forceinline__ float penalise(float x, uint32_t word, const RowRules& p) {
    if (word) {
        x *= x > 0.f ? p.inv_rep : p.rep;
        const uint32_t n = word / kGenerated;
        if (n) x -= fmaf(p.freq, (float)n, p.pres);
    }
    return x;
}

// kVec: every row of logits and out starts on 16 bytes (so that a thread reads only
// what it staged, and a mask word holds a vector's bits).
template <typename T, bool kVec, typename Word>
__global__ void __launch_bounds__(kThreads, kCtas) logit_rules_kernel(RuleArgs a) {
    // the segment's logits, its words; at the end a 32-bit word an entry for the biases
    extern __shared__ uint4 smem[];
    uint4* const staged = smem;
    uint4* const counts =
        reinterpret_cast<uint4*>(reinterpret_cast<T*>(smem) + a.segment + kSlack);
    uint32_t* const last_bias = reinterpret_cast<uint32_t*>(smem);
    const int32_t b = blockIdx.y;
    const int32_t lo = blockIdx.x * a.segment;
    const int32_t len = min(a.segment, a.vocab - lo);
    const T* row = static_cast<const T*>(a.logits) + (int64_t)b * a.stride + lo;
    float* out = a.out + (int64_t)b * a.vocab + lo;
    const uint32_t* mask = nullptr;
    const int32_t mask_words = (a.vocab + 31) / 32;
    if (a.r.allowed_mask != nullptr)
        mask = a.r.allowed_mask + (int64_t)b * mask_words + (lo >> 5);   // lo % 32 == 0

    // Rows that do not start on 16 bytes: entry i of the segment is staged at
    // in_at + i, as far from 16 bytes as it is in memory; out's first 16 bytes begin
    // with entry out_at, and the words are moved so that its word begins four.
    constexpr int E = 16 / sizeof(T);        // entries per load
    const int in_at = kVec ? 0 : (int)((uintptr_t)row % 16 / sizeof(T));
    const int out_at = kVec ? 0 : min(len, (int)(-((uintptr_t)out >> 2) & 3));
    const int word_at = kVec ? 0 : -out_at & 3;
    Word* const words = reinterpret_cast<Word*>(counts);     // entry i's at word_at + i
    T* const entries = reinterpret_cast<T*>(smem) + in_at;

    // ---- the segment's logits, all in flight while the history is counted ----
    constexpr int U = (kMaxSegment / E + kThreads - 1) / kThreads;
    const int head = kVec ? 0 : min(len, -in_at & (E - 1));  // entries ahead of 16 bytes
    const int nv = (len - head) / E;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int v = threadIdx.x + u * kThreads;
        if (v < nv) cp_async16(entries + head + v * E, row + head + v * E);
    }
    // kVec: a word of the mask a vector; else the segment's words, one a thread
    constexpr int kMaskWords = kMaxSegment / 32;
    static_assert(kMaskWords <= kThreads, "a word of the mask a thread");
    __shared__ uint32_t mask_bits[kVec ? 1 : kMaskWords + 1];
    uint32_t allow[kVec ? U : 1];
    if constexpr (kVec) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = threadIdx.x + u * kThreads;
            allow[u] = v < nv && mask ? __ldg(mask + (v * E >> 5)) : 0xffffffffu;
        }
    } else {
        const int i = threadIdx.x, j = head + nv * E + threadIdx.x;
        if (i < head) entries[i] = row[i];
        if (j < len) entries[j] = row[j];
        allow[0] = mask && i < (len + 31) / 32 ? __ldg(mask + i) : 0xffffffffu;
    }

    // the row's first tokens, before its lengths are known (the row has max_tokens
    // entries whatever they are)
    constexpr int kIds = 8;                  // loads in flight a lane
    const int32_t* ids = a.r.token_ids + (int64_t)b * a.r.max_tokens;
    int32_t first_ids[kIds];
    if (a.r.token_ids != nullptr) {
#pragma unroll
        for (int u = 0; u < kIds; ++u) {
            const int32_t i = threadIdx.x + u * kThreads;
            if (i < a.r.max_tokens) first_ids[u] = __ldg(ids + i);
        }
    }
    // the row's biases, and this thread's first one
    int32_t e0 = 0, e1 = 0, bias_id = -1;
    float bias_value = 0.f;
    if (a.r.bias_offsets != nullptr) {
        e0 = a.r.bias_offsets[b];
        e1 = a.r.bias_offsets[b + 1];
        if (e0 < 0 || e1 < e0 || e1 > a.r.num_biases) {
            if (lo == 0 && threadIdx.x == 0) pkv::report(a.status, PKV_STATUS_BAD_SEQLENS);
            e0 = e1 = 0;
        }
        if (e0 + (int)threadIdx.x < e1) {
            bias_id = __ldg(a.r.bias_token_ids + e0 + threadIdx.x);
            bias_value = __ldg(a.r.bias_values + e0 + threadIdx.x);
        }
    }

    // ---- the row's history ----
    RowRules p{1.f, 1.f, 0.f, 0.f, false};
    int32_t n_tokens = 0, n_prompt = 0;
    if (a.r.token_ids != nullptr) {
        n_tokens = a.r.max_tokens;
        // one round trip for all of them
        if (a.r.token_lens != nullptr) n_tokens = a.r.token_lens[b];
        if (a.r.prompt_lens != nullptr) n_prompt = a.r.prompt_lens[b];
        if (a.r.repetition_penalties != nullptr) p.rep = a.r.repetition_penalties[b];
        if (a.r.presence_penalties != nullptr) p.pres = a.r.presence_penalties[b];
        if (a.r.frequency_penalties != nullptr) p.freq = a.r.frequency_penalties[b];
        if (n_tokens < 0 || n_tokens > a.r.max_tokens || n_prompt < 0 || n_prompt > n_tokens) {
            if (lo == 0 && threadIdx.x == 0) pkv::report(a.status, PKV_STATUS_BAD_SEQLENS);
            n_tokens = 0;
        }
        const bool rep_ok = p.rep >= 0x1p-100f && p.rep <= 0x1p100f;     // 1 / rep is as good
        const bool add_ok = isfinite(p.freq) && isfinite(p.pres);
        if (!(rep_ok && add_ok) && lo == 0 && threadIdx.x == 0)
            pkv::report(a.status, PKV_STATUS_BAD_PENALTY);
        if (!rep_ok) p.rep = 1.f;
        p.inv_rep = __frcp_rn(p.rep);
        if (!isfinite(p.freq)) p.freq = 0.f;
        if (!isfinite(p.pres)) p.pres = 0.f;
        p.penalties = n_tokens > 0 && (p.rep != 1.f || p.freq != 0.f || p.pres != 0.f);
    }
    if (p.penalties) {
        for (int i = threadIdx.x; i < ((len + 3) * (int)sizeof(Word) + 15) / 16; i += kThreads)
            counts[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        bool bad = false;
        auto count = [&](int32_t i, int32_t id) {
            bad |= id >= a.vocab;
            const uint32_t at = (uint32_t)(id - lo);
            if (id < lo || at >= (uint32_t)len) return;
            count_token(words, at + word_at, i < n_prompt);
        };
#pragma unroll
        for (int u = 0; u < kIds; ++u) {
            const int32_t i = threadIdx.x + u * kThreads;
            if (i < n_tokens) count(i, first_ids[u]);
        }
        for (int32_t i0 = kIds * kThreads + threadIdx.x; i0 < n_tokens; i0 += kIds * kThreads) {
            int32_t id[kIds];
#pragma unroll
            for (int u = 0; u < kIds; ++u) {
                const int32_t i = i0 + u * kThreads;
                if (i < n_tokens) id[u] = __ldg(ids + i);
            }
#pragma unroll
            for (int u = 0; u < kIds; ++u)
                if (i0 + u * kThreads < n_tokens) count(i0 + u * kThreads, id[u]);
        }
        if (bad && lo == 0) pkv::report(a.status, PKV_STATUS_BAD_TOKEN_ID);
        __syncthreads();
    } else if (lo == 0 && a.status != nullptr) {
        // penalties that change nothing: the tokens are only checked
        bool bad = false;
        for (int32_t i = threadIdx.x; i < n_tokens; i += kThreads)
            bad |= __ldg(ids + i) >= a.vocab;
        if (bad) pkv::report(a.status, PKV_STATUS_BAD_TOKEN_ID);
    }

    // ---- one pass over the segment ----
    if constexpr (kVec) {
        asm volatile("cp.async.wait_all;" ::: "memory");     // this thread's own vectors
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = threadIdx.x + u * kThreads;
            if (v >= nv) continue;
            const uint4 raw = staged[v];
            const T* in = reinterpret_cast<const T*>(&raw);
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = to_float(in[e]);
            bool changed = !a.in_place;
            if (p.penalties) {
#pragma unroll
                for (int q = 0; q < E / 4; ++q) {
                    const uint4 w = four_words(words, v * E + 4 * q);
                    if ((w.x | w.y | w.z | w.w) == 0) continue;
                    changed = true;
                    x[4 * q] = penalise(x[4 * q], w.x, p);
                    x[4 * q + 1] = penalise(x[4 * q + 1], w.y, p);
                    x[4 * q + 2] = penalise(x[4 * q + 2], w.z, p);
                    x[4 * q + 3] = penalise(x[4 * q + 3], w.w, p);
                }
            }
            constexpr uint32_t kAll = (1u << E) - 1u;
            const uint32_t bits = allow[u] >> (v * E & 31) & kAll;
            if (bits != kAll) {
                changed = true;
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (!(bits >> e & 1u)) x[e] = -INFINITY;
            }
            if (changed) {
#pragma unroll
                for (int q = 0; q < E / 4; ++q)
                    *reinterpret_cast<float4*>(out + v * E + 4 * q) =
                        make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
            }
        }
        for (int i = nv * E + threadIdx.x; i < len; i += kThreads) {
            float x = to_float(row[i]);
            if (p.penalties) x = penalise(x, words[word_at + i], p);
            if (mask && !(mask[i >> 5] >> (i & 31) & 1u)) x = -INFINITY;
            out[i] = x;
        }
    } else {
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (threadIdx.x < kMaskWords) mask_bits[threadIdx.x] = allow[0];
        if (threadIdx.x == 0) mask_bits[kMaskWords] = 0xffffffffu;
        __syncthreads();                     // a vector of out lies across two of the row's
        auto bits_at = [&](int i) {          // 32 entries' bits from i on
            return __funnelshift_r(mask_bits[i >> 5], mask_bits[(i >> 5) + 1], i & 31);
        };
        const bool alike = (in_at + out_at) % 4 == 0;        // off 16 bytes by as many entries
        const int n4 = (len - out_at) / 4;
#pragma unroll 4
        for (int v = threadIdx.x; v < n4; v += kThreads) {
            const int i = out_at + 4 * v;
            float x[4];
            alignas(16) T in[4];
            if (alike) {
                using Four = std::conditional_t<sizeof(T) == 4, uint4, uint2>;
                *reinterpret_cast<Four*>(in) = *reinterpret_cast<const Four*>(entries + i);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) in[e] = entries[i + e];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = to_float(in[e]);
            bool changed = !a.in_place;
            if (p.penalties) {
                const uint4 w = four_words(words, word_at + i);
                if ((w.x | w.y | w.z | w.w) != 0) {
                    changed = true;
                    x[0] = penalise(x[0], w.x, p);
                    x[1] = penalise(x[1], w.y, p);
                    x[2] = penalise(x[2], w.z, p);
                    x[3] = penalise(x[3], w.w, p);
                }
            }
            const uint32_t bits = bits_at(i) & 15u;
            if (bits != 15u) {
                changed = true;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(bits >> e & 1u)) x[e] = -INFINITY;
            }
            if (changed) *reinterpret_cast<float4*>(out + i) = make_float4(x[0], x[1], x[2], x[3]);
        }
        // ahead of the vectors and behind them
        const int rest = out_at + len - (out_at + 4 * n4);
        if ((int)threadIdx.x < rest) {
            const int i = (int)threadIdx.x < out_at ? threadIdx.x : threadIdx.x + 4 * n4;
            float x = to_float(entries[i]);
            if (p.penalties) x = penalise(x, words[word_at + i], p);
            if (!(bits_at(i) & 1u)) x = -INFINITY;
            out[i] = x;
        }
    }

    // ---- biases of this segment's entries: the last one for a token counts ----
    if (e1 > e0) {
        // f(entry of the row, token, value) of this thread's biases
        auto each = [&](auto f) {
            if (bias_id >= 0) f((uint32_t)threadIdx.x, bias_id, bias_value);
            for (int32_t e = e0 + kThreads + threadIdx.x; e < e1; e += kThreads)
                f((uint32_t)(e - e0), __ldg(a.r.bias_token_ids + e), __ldg(a.r.bias_values + e));
        };
        auto here = [&](int32_t id) { return id >= lo && id - lo < len; };
        bool bad = false, some = false;
        each([&](uint32_t, int32_t id, float) {
            bad |= id >= a.vocab;
            some |= here(id);
        });
        if (bad && lo == 0) pkv::report(a.status, PKV_STATUS_BAD_TOKEN_ID);
        // (the barrier: the counts are read, the entries written)
        if (__syncthreads_or(some)) {
            each([&](uint32_t, int32_t id, float) {
                if (here(id)) last_bias[id - lo] = 0;
            });
            __syncthreads();
            each([&](uint32_t e, int32_t id, float) {
                if (here(id)) atomicMax(&last_bias[id - lo], e + 1);
            });
            __syncthreads();
            each([&](uint32_t e, int32_t id, float value) {
                if (!here(id) || last_bias[id - lo] != e + 1) return;
                const int i = id - lo;
                if (mask && !(mask[i >> 5] >> (i & 31) & 1u)) return;
                out[i] += value;
            });
        }
    }

    // ---- a row whose mask leaves nothing ----
    if (lo == 0 && mask != nullptr && a.status != nullptr) {
        bool any = false;
        for (int32_t w = threadIdx.x; w < mask_words; w += kThreads) {
            const int32_t left = a.vocab - w * 32;
            const uint32_t live = left >= 32 ? 0xffffffffu : (1u << left) - 1u;
            any |= (__ldg(mask + w) & live) != 0;
        }
        if (!__syncthreads_or(any) && threadIdx.x == 0)
            pkv::report(a.status, PKV_STATUS_NO_ALLOWED_TOKEN);
    }
}

template <typename T>
int launch_rules(RuleArgs& a, cudaStream_t s) {
    // Segments: 8192 entries when the rows alone fill the GPU (each segment
    // reads the whole history), less down to 1024 for a few rows, so that about
    // six CTAs an SM share the work.
    const int64_t want = (int64_t)pkv_num_sms() * 6;
    int64_t seg = ((int64_t)a.batch * a.vocab + want - 1) / want;
    seg = (seg + 1023) / 1024 * 1024;
    if (seg > kMaxSegment) seg = kMaxSegment;
    a.segment = (int32_t)seg;
    const bool vec = (((uintptr_t)a.logits | (uintptr_t)a.out) & 15) == 0 &&
                     (a.stride * (int64_t)sizeof(T)) % 16 == 0 && a.vocab % 4 == 0;
    // 16-bit words hold a count of up to 32767 tokens (with a prompt's bit)
    const bool wide = a.r.token_ids && a.r.max_tokens > 32767;
    const int smem = (a.segment + kSlack) * ((int)sizeof(T) + (wide ? 4 : 2));
    void (*const kernel)(RuleArgs) =
        vec ? wide ? logit_rules_kernel<T, true, uint32_t> : logit_rules_kernel<T, true, uint16_t>
        : wide ? logit_rules_kernel<T, false, uint32_t>
               : logit_rules_kernel<T, false, uint16_t>;
    static std::atomic<uint64_t> configured[4];
    if (!pkv_dynamic_smem_once((const void*)kernel,
                               (kMaxSegment + kSlack) * ((int)sizeof(T) + (wide ? 4 : 2)),
                               configured[vec * 2 + wide]))
        return PKV_ERR_CUDA;
    const unsigned segs = (unsigned)((a.vocab + a.segment - 1) / a.segment);
    for (int32_t b0 = 0; b0 < a.batch; b0 += 65535) {
        RuleArgs sub = a;
        const int32_t rows = a.batch - b0 < 65535 ? a.batch - b0 : 65535;
        sub.logits = (const T*)a.logits + (int64_t)b0 * a.stride;
        sub.out = a.out + (int64_t)b0 * a.vocab;
        pkv_logit_rules& r = sub.r;
        if (r.token_ids) r.token_ids += (int64_t)b0 * r.max_tokens;
        if (r.prompt_lens) r.prompt_lens += b0;
        if (r.token_lens) r.token_lens += b0;
        if (r.repetition_penalties) r.repetition_penalties += b0;
        if (r.presence_penalties) r.presence_penalties += b0;
        if (r.frequency_penalties) r.frequency_penalties += b0;
        if (r.bias_offsets) r.bias_offsets += b0;
        if (r.allowed_mask) r.allowed_mask += (int64_t)b0 * ((a.vocab + 31) / 32);
        const dim3 grid(segs, (unsigned)rows);
        kernel<<<grid, kThreads, smem, s>>>(sub);
        if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

}  // namespace

extern "C" int pkv_apply_logit_rules(const void* logits, int32_t logits_type,
                                     int64_t logits_stride, int32_t batch, int32_t vocab,
                                     pkv_logit_rules rules, float* out, uint32_t* status,
                                     void* stream) {
    if (batch < 0 || vocab <= 0 || logits_stride < vocab) return PKV_ERR_BAD_DIMENSION;
    if (logits_type != PKV_FP32 && logits_type != PKV_BF16 && logits_type != PKV_FP16)
        return PKV_ERR_UNSUPPORTED;
    if (rules.token_ids && rules.max_tokens < 0) return PKV_ERR_BAD_DIMENSION;
    if (rules.bias_offsets && rules.num_biases < 0) return PKV_ERR_BAD_DIMENSION;
    if (batch == 0) return PKV_OK;
    if (!logits || !out) return PKV_ERR_NULL_POINTER;
    if (rules.bias_offsets && rules.num_biases > 0 && (!rules.bias_token_ids || !rules.bias_values))
        return PKV_ERR_NULL_POINTER;
    const uintptr_t entry = logits_type == PKV_FP32 ? 4 : 2;
    if ((uintptr_t)logits % entry) return PKV_ERR_MISALIGNED;
    if (((uintptr_t)out | (uintptr_t)rules.token_ids | (uintptr_t)rules.prompt_lens |
         (uintptr_t)rules.token_lens | (uintptr_t)rules.repetition_penalties |
         (uintptr_t)rules.presence_penalties | (uintptr_t)rules.frequency_penalties |
         (uintptr_t)rules.bias_offsets | (uintptr_t)rules.bias_token_ids |
         (uintptr_t)rules.bias_values | (uintptr_t)rules.allowed_mask) & 3)
        return PKV_ERR_MISALIGNED;
    // in place only as a whole: fp32 rows that lie where the output's do
    const bool in_place = logits == (const void*)out;
    if (in_place && (logits_type != PKV_FP32 || (batch > 1 && logits_stride != vocab)))
        return PKV_ERR_UNSUPPORTED;
    if (!in_place) {
        const uintptr_t x0 = (uintptr_t)logits, y0 = (uintptr_t)out;
        const uintptr_t x1 = x0 + ((uintptr_t)(batch - 1) * logits_stride + vocab) * entry;
        const uintptr_t y1 = y0 + (uintptr_t)batch * vocab * 4;
        if (x0 < y1 && y0 < x1) return PKV_ERR_UNSUPPORTED;
    }
    RuleArgs a{};
    a.logits = logits;
    a.stride = logits_stride;
    a.out = out;
    a.batch = batch;
    a.vocab = vocab;
    a.r = rules;
    a.status = status;
    a.in_place = in_place;
    cudaStream_t s = (cudaStream_t)stream;
    if (logits_type == PKV_FP32) return launch_rules<float>(a, s);
    if (logits_type == PKV_BF16) return launch_rules<__nv_bfloat16>(a, s);
    return launch_rules<__half>(a, s);
}
