// Processing of logits before they are scored or sampled: penalties for repeated tokens,
// biases, grammar masks (include/lp_head.h).
//
// A thread-block cluster takes one logits row and a chunk of the vocabulary; each of its
// CTAs owns a slice of `slice` tokens. The request's history is read once per cluster:
// every CTA takes its share of the tokens and adds each to the table of the CTA that owns
// the token, in that CTA's shared memory (distributed shared memory). A table word holds
// the count in the output part and, in bit 31, whether the prompt holds the token; adds and
// ors of integers commute, so the result does not depend on their order. The CTA then
// streams its slice once: logit, table word and mask bits in, the processed value out.
// Bound by HBM: the row is read once and written once; a vector whose mask bits are all 0
// is not read.
#include "lp_head_common.h"

namespace {

using namespace lph;

constexpr uint32_t kThreads = 256;
constexpr uint32_t kCluster = 8;
constexpr uint32_t kMaxSlice = 16384;  // tokens a CTA owns: a 64 KB table, three CTAs per SM
constexpr uint32_t kMinSlice = 1024;
constexpr uint32_t kBatch = 4;         // vectors a thread has in flight
constexpr uint32_t kPrompt = 0x80000000u;

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
    uint32_t T, V, B, history_total, bias_total, mask_rows, slice, row_ctas;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Add to / or into a word of another CTA's shared memory (the same offset as `addr` here).
__device__ __forceinline__ void remote_add(uint32_t addr, uint32_t rank, uint32_t v) {
    asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
                 "red.relaxed.cluster.shared::cluster.add.u32 [ra], %2;\n\t}" ::"r"(addr), "r"(rank), "r"(v)
                 : "memory");
}
__device__ __forceinline__ void remote_or(uint32_t addr, uint32_t rank, uint32_t v) {
    asm volatile("{\n\t.reg .b32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\t"
                 "red.relaxed.cluster.shared::cluster.or.b32 [ra], %2;\n\t}" ::"r"(addr), "r"(rank), "r"(v)
                 : "memory");
}

// First index in tokens[a, b) whose value is >= v.
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* tokens, uint32_t a, uint32_t b, uint32_t v) {
    while (a < b) {
        const uint32_t mid = a + (b - a) / 2;
        if (tokens[mid] < v) a = mid + 1; else b = mid;
    }
    return a;
}

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

struct Penalty {
    float rep, freq, pres;
};
__device__ __forceinline__ float penalised(float x, uint32_t word, const Penalty& q) {
    if (word == 0) return x;
    x = x > 0.f ? __fdiv_rn(x, q.rep) : x * q.rep;
    const uint32_t count = word & ~kPrompt;
    if (count) x = x - q.freq * (float)count - q.pres;
    return x;
}

// grid: rows x chunks x kCluster CTAs
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) k_process(ProcessParams p) {
    extern __shared__ __align__(16) uint32_t table[];  // slice + 4 words
    pdl_trigger();
    const uint32_t tid = threadIdx.x, rank = cluster_rank();
    const uint32_t t = blockIdx.x / p.row_ctas;
    const uint32_t part = blockIdx.x - t * p.row_ctas;                      // CTA of the row
    const uint32_t chunk0 = (part / kCluster) * (kCluster * p.slice);  // first token of the cluster
    const uint32_t lo = chunk0 + rank * p.slice;
    const uint32_t hi = lo < p.V ? min(lo + p.slice, p.V) : lo;  // this CTA's tokens [lo, hi)
    for (uint32_t i = tid; i < p.slice / 4 + 1; i += kThreads) reinterpret_cast<uint4*>(table)[i] = make_uint4(0, 0, 0, 0);
    pdl_wait();
    const T* in = static_cast<const T*>(p.logits) + (uint64_t)t * p.stride;
    float* out = p.out + (uint64_t)t * p.out_stride;
    const uint32_t table_addr = (uint32_t)__cvta_generic_to_shared(table);
    // Table slot of token v: v - lo + pad, so that the 4 tokens of an aligned vector have an
    // aligned 16-byte group of words.
    const uint32_t pad = VEC ? (uint32_t)((reinterpret_cast<uintptr_t>(out + lo) >> 2) & 3) : 0;

    // The row's request and its parameters, checked (the same in every CTA of the cluster).
    const int b = request_of(p.row_offsets, p.B, t);
    bool bad = b < 0;
    uint32_t bad_code = LP_ERR_OFFSETS;
    Penalty q = {1.f, 0.f, 0.f};
    uint32_t h0 = 0, h1 = 0, prompt_end = 0, b0 = 0, b1 = 0;
    const uint32_t* mask = nullptr;
    if (!bad) {
        if (p.repetition) q.rep = p.repetition[b];
        if (p.frequency) q.freq = p.frequency[b];
        if (p.presence) q.pres = p.presence[b];
        if (!(q.rep > 0.f) || !isfinite(q.rep) || !isfinite(q.freq) || !isfinite(q.pres)) {
            bad = true;
            bad_code = LP_ERR_PENALTY;
        }
        if (p.history && (q.rep != 1.f || q.freq != 0.f || q.pres != 0.f)) {
            h0 = p.history_offsets[b];
            h1 = p.history_offsets[b + 1];
            if (h0 > h1 || h1 > p.history_total) { bad = true; h0 = h1 = 0; }
            prompt_end = p.prompt_lens ? p.prompt_lens[b] : 0u;
        }
        if (p.bias_tokens) {
            b0 = p.bias_offsets[b];
            b1 = p.bias_offsets[b + 1];
            if (b0 > b1 || b1 > p.bias_total) { bad = true; b0 = b1 = 0; }
        }
        if (p.mask) {
            const int64_t m = p.mask_index ? (int64_t)p.mask_index[t] : (int64_t)t;
            if (m >= (int64_t)p.mask_rows) bad = true;
            else if (m >= 0) mask = p.mask + (uint64_t)m * p.mask_stride;
        }
    }
    if (bad) {
        if (tid == 0 && part == 0) flag(p.status, bad_code);
        h0 = h1 = b0 = b1 = 0;
    }
    cluster_sync();  // every table is zero before anyone adds to it
    for (uint32_t i = rank * kThreads + tid; i < h1 - h0; i += kCluster * kThreads) {
        const uint32_t v = p.history[h0 + i];
        if (v >= p.V) {
            if (part < kCluster) flag(p.status, LP_ERR_TOKEN_RANGE);
        } else if (v >= chunk0 && v - chunk0 < kCluster * p.slice) {
            const uint32_t owner = (v - chunk0) / p.slice;
            uint32_t slot = (v - chunk0) - owner * p.slice;
            if (VEC) slot += (uint32_t)((reinterpret_cast<uintptr_t>(out + chunk0 + owner * p.slice) >> 2) & 3);
            if (i < prompt_end) remote_or(table_addr + 4 * slot, owner, kPrompt);
            else remote_add(table_addr + 4 * slot, owner, 1u);
        }
    }
    cluster_sync();  // every add is visible; no CTA reads or writes another's table after this
    if (lo >= hi) return;

    const float ninf = __int_as_float(0xff800000);
    if (bad) {
        for (uint32_t v = lo + tid; v < hi; v += kThreads) out[v] = __int_as_float(0x7fffffff);
        return;
    }
    const auto one = [&](uint32_t v) {
        const bool allowed = !mask || ((mask[v >> 5] >> (v & 31)) & 1u);
        out[v] = allowed ? penalised(to_f32(in[v]), table[v - lo + pad], q) : ninf;
    };
    if constexpr (VEC) {
        const uint32_t first = min(lo + ((4u - pad) & 3u), hi);  // first aligned vector
        const uint32_t vecs = (hi - first) / 4;
        if (tid < first - lo) one(lo + tid);
        const uint32_t last = first + 4 * vecs;
        if (tid < hi - last) one(last + tid);
        const uint4* words = reinterpret_cast<const uint4*>(table + (first - lo + pad));
        for (uint32_t i0 = tid; i0 < vecs; i0 += kBatch * kThreads) {
            // the batch's loads first (out may be logits itself, so none could move past a store)
            float4 x[kBatch];
            uint32_t bits[kBatch];
#pragma unroll
            for (uint32_t u = 0; u < kBatch; ++u) {
                const uint32_t i = i0 + u * kThreads, v = first + 4 * i;
                x[u] = make_float4(ninf, ninf, ninf, ninf);
                bits[u] = i < vecs ? 0xFu : 0u;
                if (mask && i < vecs) bits[u] = __funnelshift_r(mask[v >> 5], mask[(v + 3) >> 5], v & 31) & 0xF;
            }
#pragma unroll
            for (uint32_t u = 0; u < kBatch; ++u)
                if (bits[u]) x[u] = load4<T>(in + first + 4 * (i0 + u * kThreads));
#pragma unroll
            for (uint32_t u = 0; u < kBatch; ++u) {
                const uint32_t i = i0 + u * kThreads;
                if (i >= vecs) break;
                float4 y = x[u];
                const uint4 w = words[i];
                if (bits[u] && (w.x | w.y | w.z | w.w)) {
                    y.x = penalised(y.x, w.x, q);
                    y.y = penalised(y.y, w.y, q);
                    y.z = penalised(y.z, w.z, q);
                    y.w = penalised(y.w, w.w, q);
                }
                if (bits[u] != 0xF) {
                    y.x = bits[u] & 1 ? y.x : ninf;
                    y.y = bits[u] & 2 ? y.y : ninf;
                    y.z = bits[u] & 4 ? y.z : ninf;
                    y.w = bits[u] & 8 ? y.w : ninf;
                }
                *reinterpret_cast<float4*>(out + first + 4 * i) = y;
            }
        }
    } else {
        for (uint32_t v = lo + tid; v < hi; v += kThreads) one(v);
    }
    if (b1 > b0) {
        // The request's biases: this CTA adds those of its tokens to what it has just written
        // (ids ascend strictly, so no token has two). One CTA checks the whole list.
        if (part == 0) {
            for (uint32_t i = b0 + tid; i < b1; i += kThreads) {
                if (p.bias_tokens[i] >= p.V) flag(p.status, LP_ERR_TOKEN_RANGE);
                if (i > b0 && p.bias_tokens[i - 1] >= p.bias_tokens[i]) flag(p.status, LP_ERR_OFFSETS);
            }
        }
        const uint32_t from = lower_bound(p.bias_tokens, b0, b1, lo), to = lower_bound(p.bias_tokens, b0, b1, hi);
        __syncthreads();
        for (uint32_t i = from + tid; i < to; i += kThreads) {
            const uint32_t v = p.bias_tokens[i];
            if (v < lo || v >= hi) continue;  // only where the ids do not ascend
            if (!mask || ((mask[v >> 5] >> (v & 31)) & 1u)) out[v] += p.bias_values[i];
        }
    }
}

template <typename T>
std::atomic<uint64_t> g_smem_set[2];

template <typename T>
lp_status launch_process(const ProcessParams& p, bool vec, dim3 grid, size_t smem, lp_stream_t s) {
    void (*kernel)(ProcessParams) = vec ? k_process<T, true> : k_process<T, false>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), (kMaxSlice + 4) * 4, &g_smem_set<T>[vec])) return LP_ERR_CUDA;
    return launch(kernel, grid, kThreads, smem, s, kCluster, p);
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
    // Chunks of a row: as few as the table's size allows (each reads the history again), more
    // while the CTAs of all rows would not fill the SMs twice, down to kMinSlice tokens a CTA.
    uint64_t chunks = (V + (uint64_t)kCluster * kMaxSlice - 1) / (kCluster * kMaxSlice);
    const uint64_t want = (2ull * sms + (uint64_t)kCluster * T - 1) / ((uint64_t)kCluster * T);
    const uint64_t most = (V + (uint64_t)kCluster * kMinSlice - 1) / (kCluster * kMinSlice);
    if (chunks < want) chunks = want < most ? want : most;
    uint64_t slice = (V + chunks * kCluster - 1) / (chunks * kCluster);
    p.slice = (uint32_t)((slice + 3) / 4 * 4);
    // 4 values at a time where logits and out have their 4-value boundaries at the same tokens
    const bool vec = stride % 4 == out_stride % 4 &&
                     (reinterpret_cast<uintptr_t>(logits) / e) % 4 == (reinterpret_cast<uintptr_t>(out) / 4) % 4;
    const uint64_t ctas = chunks * kCluster * T;
    if (ctas > 0x7FFFFFFFull) return LP_ERR_SHAPE;
    p.row_ctas = (uint32_t)(chunks * kCluster);
    const dim3 grid((unsigned)ctas);
    const size_t smem = (size_t)(p.slice + 4) * 4;
    if (dtype == LP_F32) return launch_process<float>(p, vec, grid, smem, stream);
    if (dtype == LP_BF16) return launch_process<__nv_bfloat16>(p, vec, grid, smem, stream);
    return launch_process<__half>(p, vec, grid, smem, stream);
}
