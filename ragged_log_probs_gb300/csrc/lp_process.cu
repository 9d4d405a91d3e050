// Processing of logits before they are scored or sampled: penalties for repeated tokens,
// biases, grammar masks (include/lp_head.h).
//
// A CTA takes a slice of the vocabulary of one logits row. It copies the slice from logits to
// out, masked, and then corrects what differs from a copy, value by value: the tokens of the
// request's history and of its biases. For the history it keeps a table in shared memory, 16
// bits a token of the slice: the count in the output part and, in the top bit, whether the
// prompt holds it (adds and ors of integers, so their order does not matter). A first pass over
// the history counts; a second one, after the copy, takes each token's word out of the table
// (the first thread to come gets it) and applies the penalties to the one value. For a request
// whose output part could overflow 15 bits the words have 32 bits and the slice is done in two
// halves. Every CTA of a row reads the history, from L2, so slices are long: 32768 tokens.
//
// Bound by HBM: a row is read once and written once, and a vector whose mask bits are all 0 is
// not read. What had to be hidden is the time before the copy (who the row belongs to, its
// parameters, its history: a few reads that wait for each other): the slice is asked for in L2
// at the very start (256 rows of 128256 f32 without lists: 57 -> 44 us, a plain copy takes 42).
// Applying the penalties during the copy, from the table, costs every warp that holds one token
// of the history the instructions for 128 values (histories to 30,000 tokens: 83 us for the same
// rows); a cluster of CTAs that sends each token to its owner's table took 138 us.
#include "lp_head_common.h"

namespace {

using namespace lph;

constexpr uint32_t kThreads = 512;
constexpr uint32_t kMaxSlice = 32768;  // tokens of a slice: a 64 KB table, three CTAs per SM
constexpr uint32_t kMinSlice = 1024;
constexpr uint32_t kResident = 3;      // CTAs per SM
constexpr uint32_t kBatch = 4;         // vectors a thread has in flight
constexpr uint32_t kPrompt16 = 0x8000u, kPrompt32 = 0x80000000u;

struct ProcessParams {
    const void* logits;
    const uint32_t* row_offsets;
    const uint32_t* history;
    const uint32_t* history_offsets;
    const uint32_t* prompt_lens;
    const float* repetition;
    const float* frequency;
    const float* presence;
    const uint32_t* bias_tokens;
    const float* bias_values;
    const uint32_t* bias_offsets;
    const uint32_t* mask;
    const int32_t* mask_index;
    float* out;
    uint32_t* status;
    uint64_t stride, out_stride, mask_stride;
    uint32_t T, V, B, history_total, bias_total, mask_rows, slice, slices;
};

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack2(w.x, __nv_bfloat16()), b = unpack2(w.y, __nv_bfloat16());
    return make_float4(a.x, a.y, b.x, b.y);
}
template <>
__device__ __forceinline__ float4 load4<__half>(const __half* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack2(w.x, __half()), b = unpack2(w.y, __half());
    return make_float4(a.x, a.y, b.x, b.y);
}

// x / rep is taken as x times the rounded 1 / rep: one rounding more than a division, which
// costs about ten instructions.
struct Penalty {
    float rep, inv, freq, pres;
};
__device__ __forceinline__ float penalised(float x, uint32_t count, const Penalty& q) {  // a token of the history
    const float y = x * (x > 0.f ? q.inv : q.rep);
    return count ? y - q.freq * (float)count - q.pres : y;
}

// What a row needs, in shared memory: its request, checked, and the request's parameters.
struct Row {
    int32_t request;         // -1: the row's values are NaN
    uint32_t counted;        // the history has an effect
    int64_t mask;            // first word of the row's mask, -1: none
    uint32_t h0, h1, prompt; // its history, and how much of that is the prompt
    uint32_t b0, b1;         // its biases
    Penalty q;
};

// The request of row t, found by one warp: 32 offsets at a time, the row's own number first
// (a request a row). off[0] <= t < off[B] or -1; ends for any contents of off.
__device__ __forceinline__ int32_t request_by_warp(const uint32_t* off, uint32_t B, uint32_t t) {
    if (!off) return (int32_t)t;
    const uint32_t lane = threadIdx.x & 31, guess = min(t, B - 1);
    const uint32_t probe = off[lane == 0 ? guess : lane == 1 ? guess + 1 : lane == 2 ? 0 : B];
    const uint32_t at = __shfl_sync(0xFFFFFFFFu, probe, 0), after = __shfl_sync(0xFFFFFFFFu, probe, 1);
    if (at <= t && t < after) return (int32_t)guess;
    if (__shfl_sync(0xFFFFFFFFu, probe, 2) > t || __shfl_sync(0xFFFFFFFFu, probe, 3) <= t) return -1;
    uint32_t lo = 0, n = B;  // off[lo] <= t < off[lo + n]
    while (n > 1) {
        const uint32_t step = (n + 31) / 32, i = lane * step;
        const uint32_t below = __ballot_sync(0xFFFFFFFFu, i < n && off[lo + (i < n ? i : 0)] <= t);
        const uint32_t k = 31 - __clz(below | 1u);  // the last probe that is not past t
        lo += k * step;
        n = min(step, n - k * step);
    }
    return (int32_t)lo;
}

// One warp describes row t; loads that do not need each other's values are started together.
__device__ __forceinline__ void describe(const ProcessParams& p, uint32_t t, Row* row, bool report) {
    const uint32_t lane = threadIdx.x & 31;
    const int64_t m = !p.mask ? -1 : p.mask_index ? (int64_t)p.mask_index[t] : (int64_t)t;
    const int32_t b = request_by_warp(p.row_offsets, p.B, t);
    if (lane != 0) return;
    Row r = {b, 0u, -1, 0u, 0u, 0u, 0u, 0u, {1.f, 1.f, 0.f, 0.f}};
    uint32_t code = LP_ERR_OFFSETS;
    if (b >= 0) {
        if (p.repetition) r.q.rep = p.repetition[b];
        if (p.frequency) r.q.freq = p.frequency[b];
        if (p.presence) r.q.pres = p.presence[b];
        if (p.history) {
            r.h0 = p.history_offsets[b];
            r.h1 = p.history_offsets[b + 1];
            if (p.prompt_lens) r.prompt = p.prompt_lens[b];
        }
        if (p.bias_tokens) {
            r.b0 = p.bias_offsets[b];
            r.b1 = p.bias_offsets[b + 1];
        }
        const bool neutral = r.q.rep == 1.f && r.q.freq == 0.f && r.q.pres == 0.f;
        r.counted = !neutral && r.h1 > r.h0;
        if ((!neutral && (r.h0 > r.h1 || r.h1 > p.history_total)) || r.b0 > r.b1 || r.b1 > p.bias_total) r.request = -1;
        r.q.inv = 1.f / r.q.rep;
        if (!(r.q.rep >= LP_MIN_REPETITION && r.q.rep <= LP_MAX_REPETITION) || !isfinite(r.q.freq) || !isfinite(r.q.pres)) {
            r.request = -1;
            code = LP_ERR_PENALTY;
        }
        if (m >= (int64_t)p.mask_rows) r.request = -1;
        else if (m >= 0) r.mask = m * (int64_t)p.mask_stride;
        if (r.prompt > r.h1 - r.h0) r.prompt = r.h1 - r.h0;
    }
    if (r.request < 0 && report) flag(p.status, code);
    *row = r;
}

// Every token of h[0, n), four at a time; returns whether one of this thread's is >= limit.
template <typename F>
__device__ __forceinline__ bool each_token(const uint32_t* h, uint32_t n, uint32_t limit, F use) {
    const uint32_t head = min(n, (uint32_t)(-(reinterpret_cast<uintptr_t>(h) >> 2) & 3));  // to a 16-byte boundary
    const uint32_t quads = (n - head) / 4, last = head + 4 * quads;
    uint32_t most = 0;
    if (threadIdx.x < head) { const uint32_t v = h[threadIdx.x]; use(v); most = v; }
    if (threadIdx.x < n - last) { const uint32_t v = h[last + threadIdx.x]; use(v); most = max(most, v); }
    const uint4* h4 = reinterpret_cast<const uint4*>(h + head);
#pragma unroll 4
    for (uint32_t k = threadIdx.x; k < quads; k += kThreads) {
        const uint4 v = h4[k];
        use(v.x);
        use(v.y);
        use(v.z);
        use(v.w);
        most = max(most, max(max(v.x, v.y), max(v.z, v.w)));
    }
    return most >= limit;
}

// The table of tokens [lo, lo + size): a word of 16 bits (WIDE: 32) a token.
template <bool WIDE>
struct Table {
    uint32_t* words;
    uint32_t lo, size;
    __device__ __forceinline__ uint32_t shift(uint32_t slot) const { return WIDE ? 0 : slot % 2 * 16; }
    __device__ __forceinline__ uint32_t* word(uint32_t slot) const { return words + (WIDE ? slot : slot / 2); }

    // Count the row's history; returns whether a token was past the vocabulary.
    __device__ __forceinline__ bool count(const ProcessParams& p, const Row& row) const {
        const uint32_t* h = p.history + row.h0;
        const bool in_prompt = each_token(h, row.prompt, p.V, [&](uint32_t v) {
            if (v - lo < size) atomicOr(word(v - lo), (WIDE ? kPrompt32 : kPrompt16) << shift(v - lo));
        });
        const bool in_output = each_token(h + row.prompt, row.h1 - row.h0 - row.prompt, p.V, [&](uint32_t v) {
            if (v - lo < size) atomicAdd(word(v - lo), 1u << shift(v - lo));
        });
        return in_prompt || in_output;
    }
    // Give each token's word to one thread: use(token, in prompt, count). Empties the table.
    template <typename F>
    __device__ __forceinline__ void take(const ProcessParams& p, const Row& row, F use) const {
        (void)each_token(p.history + row.h0, row.h1 - row.h0, p.V, [&](uint32_t v) {
            const uint32_t slot = v - lo;
            if (slot >= size) return;
            const uint32_t all = WIDE ? 0xFFFFFFFFu : 0xFFFFu;
            if (!(*static_cast<volatile uint32_t*>(word(slot)) & all << shift(slot))) return;  // taken
            const uint32_t w = atomicAnd(word(slot), ~(all << shift(slot))) >> shift(slot) & all;
            if (w) use(v, w & ~(WIDE ? kPrompt32 : kPrompt16));
        });
    }
};

// Ask for a row's slice in L2.
template <typename T>
__device__ __forceinline__ void prefetch_slice(const T* row, uint32_t lo, uint32_t hi) {
    constexpr uint32_t kPiece = 4096;
    const uintptr_t from = (reinterpret_cast<uintptr_t>(row + lo) + 15) & ~(uintptr_t)15;
    const uintptr_t to = reinterpret_cast<uintptr_t>(row + hi) & ~(uintptr_t)15;
    for (uintptr_t at = from + threadIdx.x * kPiece; at < to; at += kThreads * kPiece) {
        const uint32_t bytes = to - at < kPiece ? (uint32_t)(to - at) : kPiece;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
    }
}

// grid: T x slices CTAs
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, kResident) k_process(ProcessParams p) {
    extern __shared__ __align__(16) uint32_t table[];  // slice / 2 words
    __shared__ Row s_row;
    __shared__ uint32_t s_mask[kMaxSlice / 32 + 2];    // mask words of the slice
    pdl_trigger();
    const uint32_t tid = threadIdx.x;
    const uint32_t t = blockIdx.x / p.slices, part = blockIdx.x - t * p.slices;
    const uint32_t lo = part * p.slice, hi = min(lo + p.slice, p.V);  // this CTA's tokens
    const T* in = static_cast<const T*>(p.logits) + (uint64_t)t * p.stride;
    float* out = p.out + (uint64_t)t * p.out_stride;
    const float ninf = __int_as_float(0xff800000);
    if (p.history)
        for (uint32_t i = tid; i < (p.slice + 7) / 8; i += kThreads) reinterpret_cast<uint4*>(table)[i] = make_uint4(0, 0, 0, 0);
    pdl_wait();
    if (!p.mask) prefetch_slice(in, lo, hi);
    if (tid < 32) describe(p, t, &s_row, part == 0);
    __syncthreads();
    const Row row = s_row;
    if (row.request < 0) {
        for (uint32_t v = lo + tid; v < hi; v += kThreads) out[v] = __int_as_float(0x7fffffff);
        return;
    }
    const bool masked = row.mask >= 0;
    const uint32_t word0 = lo >> 5, words = ((hi - 1) >> 5) - word0 + 1;
    if (masked) {
        for (uint32_t i = tid; i <= words; i += kThreads)  // (the last is read beside the one before)
            s_mask[i] = i < words ? p.mask[row.mask + word0 + i] : 0u;
    } else if (p.mask) {
        prefetch_slice(in, lo, hi);
    }
    const auto allowed = [&](uint32_t v) { return !masked || ((s_mask[(v >> 5) - word0] >> (v & 31)) & 1u); };
    // 15 bits hold any count of an output part of up to 32767 tokens
    const bool wide = row.counted && row.h1 - row.h0 - row.prompt > 0x7FFFu;
    const Table<false> counts = {table, lo, hi - lo};
    if (row.counted && !wide && counts.count(p, row) && part == 0) flag(p.status, LP_ERR_TOKEN_RANGE);
    // this thread's first bias, long before it is needed
    const bool biased = row.b1 - row.b0 > tid;
    const uint32_t bias_at = biased ? p.bias_tokens[row.b0 + tid] : 0u;
    const float bias = biased ? p.bias_values[row.b0 + tid] : 0.f;
    if (masked) __syncthreads();

    // the copy
    const uint32_t first = VEC ? min(lo + ((-(uint32_t)(reinterpret_cast<uintptr_t>(out + lo) >> 2)) & 3u), hi) : hi;
    const uint32_t vecs = (hi - first) / 4, vec_end = first + 4 * vecs;
    for (uint32_t v = lo + tid; v < first; v += kThreads) out[v] = allowed(v) ? to_f32(in[v]) : ninf;
    for (uint32_t v = vec_end + tid; v < hi; v += kThreads) out[v] = allowed(v) ? to_f32(in[v]) : ninf;
    if constexpr (VEC) {
        const T* in4 = in + first;
        float4* out4 = reinterpret_cast<float4*>(out + first);
        for (uint32_t i0 = tid; i0 < vecs; i0 += kBatch * kThreads) {
            // a batch's loads before its stores: out may be logits
            float4 x[kBatch];
            uint32_t bits[kBatch];
#pragma unroll
            for (uint32_t u = 0; u < kBatch; ++u) {
                const uint32_t i = i0 + u * kThreads, v = first + 4 * i;
                bits[u] = i < vecs ? 0xFu : 0u;
                if (masked && i < vecs) {
                    const uint32_t* m = s_mask + ((v >> 5) - word0);
                    bits[u] = __funnelshift_r(m[0], m[1], v & 31) & 0xF;
                }
                x[u] = make_float4(ninf, ninf, ninf, ninf);
                if (bits[u]) x[u] = load4<T>(in4 + 4 * i);
            }
#pragma unroll
            for (uint32_t u = 0; u < kBatch; ++u) {
                const uint32_t i = i0 + u * kThreads;
                if (i >= vecs) break;
                float4 y = x[u];
                if (masked) {
                    y.x = bits[u] & 1 ? y.x : ninf;
                    y.y = bits[u] & 2 ? y.y : ninf;
                    y.z = bits[u] & 4 ? y.z : ninf;
                    y.w = bits[u] & 8 ? y.w : ninf;
                }
                out4[i] = y;
            }
        }
    }

    // the history's tokens
    const auto correct = [&](uint32_t v, uint32_t count) {
        if (allowed(v)) out[v] = penalised(out[v], count, row.q);
    };
    if (row.counted && !wide) {
        __syncthreads();
        counts.take(p, row, correct);
    } else if (row.counted) {
        const uint32_t half = (p.slice + 7) / 8 * 4;  // (a table of 16 bits a token holds half as many of 32)
        for (uint32_t from = lo; from < hi; from += half) {
            const Table<true> part_counts = {table, from, min(half, hi - from)};
            const bool outside = part_counts.count(p, row);
            if (outside && part == 0 && from == lo) flag(p.status, LP_ERR_TOKEN_RANGE);
            __syncthreads();
            part_counts.take(p, row, correct);
            __syncthreads();
        }
    }
    // the biases: no token has two
    if (row.b1 > row.b0) {
        __syncthreads();
        if (biased && bias_at - lo < hi - lo && allowed(bias_at)) out[bias_at] += bias;
        for (uint32_t i = row.b0 + tid + kThreads; i < row.b1; i += kThreads) {
            const uint32_t v = p.bias_tokens[i];
            if (v - lo < hi - lo && allowed(v)) out[v] += p.bias_values[i];
        }
        if (part == 0) {  // one CTA of a row checks the list
            for (uint32_t i = row.b0 + tid; i < row.b1; i += kThreads) {
                if (p.bias_tokens[i] >= p.V) flag(p.status, LP_ERR_TOKEN_RANGE);
                if (i > row.b0 && p.bias_tokens[i - 1] >= p.bias_tokens[i]) flag(p.status, LP_ERR_OFFSETS);
            }
        }
    }
}

template <typename T>
std::atomic<uint64_t> g_smem_set[2];

template <typename T>
lp_status launch_process(const ProcessParams& p, bool vec, unsigned ctas, lp_stream_t s) {
    void (*kernel)(ProcessParams) = vec ? k_process<T, true> : k_process<T, false>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), kMaxSlice * 2, &g_smem_set<T>[vec])) return LP_ERR_CUDA;
    return launch(kernel, dim3(ctas), kThreads, (size_t)p.slice * 2, s, 1, p);
}

}  // namespace

extern "C" lp_status lp_head_process(const void* logits, uint32_t dtype, uint32_t T, uint32_t V, uint64_t stride,
                                     const uint32_t* row_offsets, uint32_t B, const uint32_t* history,
                                     const uint32_t* history_offsets, uint32_t history_total,
                                     const uint32_t* prompt_lens, const float* repetition, const float* frequency,
                                     const float* presence, const uint32_t* bias_tokens, const float* bias_values,
                                     const uint32_t* bias_offsets, uint32_t bias_total, const uint32_t* mask,
                                     uint64_t mask_stride, uint32_t mask_rows, const int32_t* mask_index, float* out,
                                     uint64_t out_stride, void* workspace, size_t workspace_bytes,
                                     lp_stream_t stream) {
    if (!logits || !out || (history && !history_offsets) ||
        (bias_tokens && (!bias_values || !bias_offsets)))
        return LP_ERR_NULL;
    if (!workspace || workspace_bytes < kHeaderBytes || !aligned_to(workspace, 256)) return LP_ERR_WORKSPACE;
    if (dtype > LP_F16) return LP_ERR_DTYPE;
    if (T == 0 || V == 0 || B == 0 || V >= 0x7FFFFFFFu || stride < V || out_stride < V)
        return LP_ERR_SHAPE;
    if (!row_offsets && B != T) return LP_ERR_SHAPE;
    if (mask && (mask_rows == 0 || mask_rows > 0x7FFFFFFFu || mask_stride < ((uint64_t)V + 31) / 32 ||
                 (!mask_index && mask_rows < T)))
        return LP_ERR_SHAPE;
    const size_t e = dtype_bytes(dtype);
    if (!aligned_to(logits, e) || !aligned_to(out, 4)) return LP_ERR_SHAPE;
    if (static_cast<const void*>(out) == logits && (dtype != LP_F32 || stride != out_stride)) return LP_ERR_SHAPE;
    const int sms = sm_count();
    if (sms == 0) return LP_ERR_CUDA;
    ProcessParams p;
    p.logits = logits;
    p.row_offsets = row_offsets;
    p.history = history_total ? history : nullptr;
    p.history_offsets = history_offsets;
    p.prompt_lens = prompt_lens;
    p.repetition = repetition;
    p.frequency = frequency;
    p.presence = presence;
    p.bias_tokens = bias_total ? bias_tokens : nullptr;
    p.bias_values = bias_values;
    p.bias_offsets = bias_offsets;
    p.mask = mask;
    p.mask_index = mask_index;
    p.out = out;
    p.status = static_cast<uint32_t*>(workspace);
    p.stride = stride;
    p.out_stride = out_stride;
    p.mask_stride = mask_stride;
    p.T = T;
    p.V = V;
    p.B = B;
    p.history_total = history_total;
    p.bias_total = bias_total;
    p.mask_rows = mask_rows;
    // Slices: as few as the table allows, up to twice as many where the last wave of CTAs is then
    // fuller (each slice more reads the history once more: 1/32 of the time is allowed for it),
    // and as many as fill the SMs where there are few rows.
    const uint64_t room = (uint64_t)sms * kResident, least = (V + (uint64_t)kMaxSlice - 1) / kMaxSlice;
    uint64_t slices = least;
    if (T * least < room) {
        const uint64_t most = (V + (uint64_t)kMinSlice - 1) / kMinSlice;
        slices = room / T < most ? room / T : most;
        if (slices < least) slices = least;
    } else {
        const auto cost = [&](uint64_t n) {  // waves, by the length of a slice and a part for the history
            return (double)((T * n + room - 1) / room) * (1.0 / (double)n + 1.0 / 32.0 / (double)least);
        };
        for (uint64_t n = least + 1; n <= 2 * least; ++n)
            if (cost(n) < cost(slices)) slices = n;
    }
    p.slice = (uint32_t)(((V + slices - 1) / slices + 7) / 8 * 8);
    p.slices = (V + p.slice - 1) / p.slice;
    // 4 values at a time where logits and out have their 4-value boundaries at the same tokens
    const bool vec = stride % 4 == out_stride % 4 &&
                     (reinterpret_cast<uintptr_t>(logits) / e) % 4 == (reinterpret_cast<uintptr_t>(out) / 4) % 4;
    const uint64_t ctas = (uint64_t)p.slices * T;
    if (ctas > 0x7FFFFFFFull) return LP_ERR_SHAPE;
    if (dtype == LP_F32) return launch_process<float>(p, vec, (unsigned)ctas, stream);
    if (dtype == LP_BF16) return launch_process<__nv_bfloat16>(p, vec, (unsigned)ctas, stream);
    return launch_process<__half>(p, vec, (unsigned)ctas, stream);
}
