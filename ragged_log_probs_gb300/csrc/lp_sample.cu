// Draw of the next token (include/lp_head.h): temperature, top-k, top-p and min-p, from a given
// random number a row.
//
// A row belongs to a cluster of up to eight CTAs, each with a slice of it in shared memory, read
// from HBM once. Weights exp((x - max) / tau) are formed with about 40 correct bits (a table of 64
// powers and a short series, in pairs of f32) and added as pairs or as integers of 2^-43: the token
// is a comparison of sums of up to some hundred thousand weights with each other, and f32's
// rounding would move it in a few rows of a hundred. All three filters keep a prefix of the order
// (value descending, id ascending), so that what is kept is told by the last kept (value, id):
//   top-k: a bound below the k-th value is read from a coarse histogram of the threads' largest;
//          what lies above it is listed and sorted by the cluster's first CTA.
//   top-p: what weighs less than (1 - p) Z / V is never kept; what is left is listed and sorted
//          when it is short, else a histogram over the values' bits finds the bin in which p Z
//          is reached, and that bin is listed. A bin of more than fits is cut again; one that
//          holds a single value is cut by id.
// The draw follows the ids: the kept weights are summed by warp, the warp in which u Z falls
// walks its part once more.
#include <cooperative_groups.h>

#include "lp_head_common.h"

namespace {

using namespace lph;
namespace cg = cooperative_groups;

constexpr uint32_t kThreads = 512, kWarps = kThreads / 32;
constexpr uint32_t kMaxCluster = 8;
constexpr uint32_t kList = 1024;   // tokens that are sorted
constexpr uint32_t kBins = kThreads;
constexpr uint32_t kBound = 256;
constexpr uint32_t kTable = 64;
constexpr uint32_t kLowest = 0x00800000u;  // ordered() of the lowest finite value
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kPoint = 43;         // weights as integers: 2^43 is that of the largest
constexpr float kSmallest = -40.f; // log2 of the smallest weight that counts
constexpr uint32_t kMaxSlice = LP_MAX_SAMPLE_VOCAB / kMaxCluster;
static_assert(LP_MAX_SAMPLE_VOCAB % (kMaxCluster * kThreads * 8) == 0, "whole rounds, and one for unaligned rows");

struct SampleParams {
    const void* logits;
    const float* uniform;
    const uint32_t* row_offsets;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    uint32_t* out;
    float* out_logprob;
    uint32_t* status;
    uint64_t stride;
    uint32_t T, V, B;
    uint32_t chunk;  // elements of a warp: whole vectors of 32 lanes
};

// A value's bits in the order of the values (both zeros were made one before).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// The coarse bins of the values: eight to an octave from 2^-3 to 2^13 on both sides of 0.
__device__ __forceinline__ uint32_t bound_bin(float x) {
    const uint32_t a = (__float_as_uint(x) & 0x7FFFFFFFu) >> 20;
    const uint32_t i = min(max(a, 992u) - 992u, 127u);
    return x < 0.f ? 127 - i : 128 + i;
}
__device__ __forceinline__ uint32_t bound_edge(uint32_t bin) {  // ordered() of the least value in it
    if (bin > 128) return ordered(__uint_as_float((bin - 128 + 992) << 20));
    if (bin == 128) return ordered(0.f);
    return bin == 0 ? kLowest : ordered(-__uint_as_float(((993 + 127 - bin) << 20) - 1));
}

// What a row is drawn with.
struct Setting {
    uint32_t ok;           // 0: no token
    float tau, chi, clo;   // chi + clo = log2(e) / tau
    float top_p, u;
    double log_min_p;      // -inf: off
    uint32_t k;            // 0: off
};

struct Cut {
    uint32_t key, id;      // kept: a larger key, or this one with an id up to this
    uint32_t again;        // the search goes on among keys above `above`, for the weight `target`
    uint32_t above;
    uint64_t target;
};

struct Shared {
    uint64_t list[kList];   // key << 32 | ~id
    uint64_t weight[kList];
    union {
        struct {
            uint32_t count[kBins], low[kBins], high[kBins];
        };
        uint32_t key[kList];
    };
    uint64_t scan[kWarps];
    uint64_t warp_sum[kWarps];
    uint32_t warp_count[kWarps];
    float warp_max[kWarps];
    float2 table[kTable];
    uint32_t bound[kBound];
    Setting set;
    Cut cut;
    float cta_max;
    uint64_t cta_sum;
    uint32_t listed;
    uint32_t found_bin, found_count;     // of a histogram
    uint64_t found_before;
    uint32_t found_before_count;
    uint64_t words[4];
};

// 2^(j / 64) as a pair of f32, made from double's exp2.
__device__ __forceinline__ float2 table_entry(uint32_t j) {
    const double t = exp2((double)j * (1.0 / kTable));
    const float h = (float)t;
    return make_float2(h, (float)(t - (double)h));
}

struct Weight {
    float hi, lo;  // hi + lo, hi rounded to 24 bits
};
// exp((x - m) / tau); 0 below 2^-40.
__device__ __forceinline__ Weight weigh(float x, float m, float chi, float clo, const float2* table) {
    const float d = x - m, back = d - x, err = (x - (d - back)) + (-m - back);
    const float p = d * chi;
    const float rest = fmaf(err, chi, fmaf(d, clo, fmaf(d, chi, -p)));
    if (!(p + rest >= kSmallest)) return {0.f, 0.f};
    constexpr float kMagic = 196608.f;  // 1.5 * 2^17: a unit in the last place is 1 / 64
    const float r = p + kMagic;
    const int k = (int)(__float_as_uint(r) - 0x48400000u);
    const float g = (p - (r - kMagic)) + rest;  // |g| <= 1 / 128
    // 2^g - 1 = g ln 2 + (g ln 2)^2 / 2 + ...; the first term as a pair
    constexpr float kL1 = 0.693147180559945f, kL2 = -1.9046542e-9f;
    const float qh = g * kL1;
    float ql = fmaf(g, kL2, fmaf(g, kL1, -qh));
    ql = fmaf(g * g, fmaf(g, fmaf(g, 0.00961812910762848f, 0.0555041086648216f), 0.240226506959101f), ql);
    const float2 t = table[k & (kTable - 1)];
    const float a = t.x * qh, b = fmaf(t.x, qh, -a);
    const float s = t.x + a;
    const float e = ((t.x - s) + a) + (fmaf(t.x, ql, t.y) + fmaf(t.y, qh, b));
    const float scale = __uint_as_float((uint32_t)((k >> 6) + 127) << 23);
    return {s * scale, e * scale};
}
__device__ __forceinline__ uint64_t fixed(Weight w) {
    return __float2ull_rn(w.hi * 8796093022208.f) + (uint64_t)__float2ll_rn(w.lo * 8796093022208.f);  // 2^43
}
// Sums of weights, as a pair.
__device__ __forceinline__ void add(Weight& s, Weight w) {
    const float t = s.hi + w.hi, z = t - s.hi;
    s.lo += ((s.hi - (t - z)) + (w.hi - z)) + w.lo;
    s.hi = t;
}

// floor(f z) for f in 0..1, and whether that is exact.
__device__ __forceinline__ uint64_t part_of(float f, uint64_t z, bool* exact) {
    const uint32_t b = __float_as_uint(f), e = b >> 23;
    const uint64_t mant = e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
    const int shift = 150 - (int)(e ? e : 1);  // f = mant 2^-shift, shift >= 23
    const uint64_t lo = mant * z, hi = __umul64hi(mant, z);
    if (shift >= 128) {
        *exact = (lo | hi) == 0;
        return 0;
    }
    if (shift >= 64) {
        const int s = shift - 64;
        *exact = lo == 0 && (s == 0 || (hi & ((1ull << s) - 1)) == 0);
        return hi >> s;
    }
    *exact = (lo & ((1ull << shift) - 1)) == 0;
    return lo >> shift | hi << (64 - shift);
}
__device__ __forceinline__ uint64_t reached_at(float p, uint64_t z) {  // the least sum that is not below p z, at least 1
    bool exact;
    const uint64_t t = part_of(p, z, &exact);
    return max(exact ? t : t + 1, (uint64_t)1);
}

__device__ __forceinline__ uint64_t warp_scan(uint64_t v) {  // inclusive
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
        const uint64_t o = __shfl_up_sync(0xFFFFFFFFu, v, k);
        if (lane >= k) v += o;
    }
    return v;
}
// Inclusive scan over the CTA's threads.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* scratch) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_scan(v);
    __syncthreads();
    if (lane == 31) scratch[warp] = v;
    __syncthreads();
    uint64_t before = 0;
#pragma unroll
    for (uint32_t k = 0; k < kWarps; ++k) before += k < warp ? scratch[k] : 0;
    return v + before;
}

// n keys (n <= kList) in descending order; what follows up to the next power of two becomes 0.
__device__ __forceinline__ void sort_list(uint64_t* list, uint32_t n) {
    uint32_t size = 2;
    while (size < n) size *= 2;
    for (uint32_t i = n + threadIdx.x; i < size; i += kThreads) list[i] = 0;
    __syncthreads();
    for (uint32_t k = 2; k <= size; k *= 2)
        for (uint32_t j = k / 2; j > 0; j /= 2) {
            const uint32_t t = threadIdx.x;
            if (t < size / 2) {
                const uint32_t i = 2 * j * (t / j) + t % j;
                const uint64_t a = list[i], b = list[i + j];
                if ((a < b) == ((i & k) == 0)) {
                    list[i] = b;
                    list[i + j] = a;
                }
            }
            __syncthreads();
        }
}

// Vectors of 16 bytes.
template <typename T>
struct Vec {
    static constexpr uint32_t kElems = 16 / sizeof(T);
};
__device__ __forceinline__ void widen(uint4 w, float (&v)[4], float) {
    v[0] = __uint_as_float(w.x) + 0.f;  // (-0 becomes 0)
    v[1] = __uint_as_float(w.y) + 0.f;
    v[2] = __uint_as_float(w.z) + 0.f;
    v[3] = __uint_as_float(w.w) + 0.f;
}
template <typename T>
__device__ __forceinline__ void widen(uint4 w, float (&v)[8], T) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(u[i], T());
        v[2 * i] = f.x + 0.f;
        v[2 * i + 1] = f.y + 0.f;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(const SampleParams p) {
    constexpr uint32_t VEC = Vec<T>::kElems;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ Shared sh;
    uint4* slice = reinterpret_cast<uint4*>(smem_raw);
    const cg::cluster_group cluster = cg::this_cluster();
    const uint32_t C = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t row = blockIdx.x / C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_trigger();
    for (uint32_t i = threadIdx.x; i < kTable; i += kThreads) sh.table[i] = table_entry(i);
    for (uint32_t i = threadIdx.x; i < kBound; i += kThreads) sh.bound[i] = 0;
    if (threadIdx.x == 0) sh.listed = 0;
    pdl_wait();

    // The row in units of aligned vectors: element i of the row is number i + before. Slices and the
    // warps' parts of them are whole vectors; what lies outside the row becomes -inf.
    const T* x = static_cast<const T*>(p.logits) + (uint64_t)row * p.stride;
    const uint32_t before = (uint32_t)(reinterpret_cast<uintptr_t>(x) / sizeof(T)) % VEC;
    const uint32_t vecs = p.chunk / VEC;                       // of a warp
    const uint32_t first = (rank * kWarps + warp) * p.chunk;   // number of the warp's first element
    uint4* mine = slice + warp * vecs;
    const auto id_of = [&](uint32_t vec, uint32_t i) { return first + vec * VEC + i - before; };

    // The setting, by one thread, while the others read.
    if (threadIdx.x == kThreads - 32) {
        Setting s = {};
        const int b = request_of(p.row_offsets, p.B, row);
        s.ok = b >= 0;
        if (b < 0) {
            if (rank == 0) flag(p.status, LP_ERR_OFFSETS);
        } else {
            float tau = p.temperature ? p.temperature[b] : 1.f, top_p = p.top_p ? p.top_p[b] : 1.f;
            const float min_p = p.min_p ? p.min_p[b] : 0.f, u = p.uniform[row];
            const int k = p.top_k ? p.top_k[b] : 0;
            if (!(tau >= 0.f && tau <= 3.402823466e38f)) {
                s.ok = 0;
                if (rank == 0) flag(p.status, LP_ERR_TEMPERATURE);
            }
            if (!(top_p >= 0.f && top_p <= 1.f) || !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f)) {
                s.ok = 0;
                if (rank == 0) flag(p.status, LP_ERR_SAMPLING);
            }
            s.k = k > 0 && (uint32_t)k < p.V ? (uint32_t)k : 0;
            if (tau == 0.f) {
                tau = 1.f;
                s.k = 1;
            }
            const double c = 1.4426950408889634 / (double)tau;
            s.tau = tau;
            s.chi = (float)c;
            s.clo = (float)(c - (double)s.chi);
            s.top_p = top_p;
            s.u = u;
            s.log_min_p = min_p > 0.f ? log((double)min_p) : -(double)__uint_as_float(0x7F800000u);
        }
        sh.set = s;
    }

    // ---- 1. read, largest value, threads' largest in coarse bins
    float top = -__uint_as_float(0x7F800000u);
#pragma unroll 4
    for (uint32_t v = lane; v < vecs; v += 32) {
        const uint32_t at = first + v * VEC;
        uint4 w;
        if (at >= before && at + VEC <= p.V + before) {
            w = *reinterpret_cast<const uint4*>(x + (at - before));
        } else {
            T e[VEC];
#pragma unroll
            for (uint32_t i = 0; i < VEC; ++i) {
                const uint32_t n = at + i;
                e[i] = n >= before && n < p.V + before ? x[n - before] : from_f32<T>(-__uint_as_float(0x7F800000u));
            }
            memcpy(&w, e, 16);
        }
        mine[v] = w;
        float f[VEC];
        widen(w, f, T());
#pragma unroll
        for (uint32_t i = 0; i < VEC; ++i) top = max_nan(top, f[i]);
    }
    __syncthreads();  // bins cleared
    if (top > -__uint_as_float(0x7F800000u)) atomicAdd(&sh.bound[bound_bin(top)], 1);
#pragma unroll
    for (int k = 16; k > 0; k /= 2) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
    if (lane == 0) sh.warp_max[warp] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (uint32_t k = 1; k < kWarps; ++k) top = max_nan(top, sh.warp_max[k]);
        sh.cta_max = top;
    }
    cluster.sync();
    float m = -__uint_as_float(0x7F800000u);
    for (uint32_t k = 0; k < C; ++k) m = max_nan(m, *cluster.map_shared_rank(&sh.cta_max, k));
    const Setting set = sh.set;
    const bool finite = m > -__uint_as_float(0x7F800000u) && m < __uint_as_float(0x7F800000u);
    if (!set.ok || !finite) {
        if (rank == 0 && threadIdx.x == 0) {
            if (set.ok) flag(p.status, LP_ERR_LOGITS);
            p.out[row] = kAll;
            if (p.out_logprob) p.out_logprob[row] = __uint_as_float(0x7FC00000u);
        }
        cluster.sync();  // (its largest value has been read)
        return;
    }
    const auto weight_of = [&](float f) { return weigh(f, m, set.chi, set.clo, sh.table); };
    // min-p: the least value kept
    uint32_t least = kLowest;
    if (set.log_min_p > -1e300) {
        const double want = (double)m + (double)set.tau * set.log_min_p;
        float f = (float)want;
        if (want < -3.402823466e38) f = -3.402823466e38f;
        uint32_t key = ordered(f + 0.f);
        if ((double)f < want) ++key;  // the next value up
        least = min(max(key, kLowest), ordered(m));
    }
    const auto token_is = [&](uint32_t id, float value, uint64_t z) {
        p.out[row] = id;
        if (p.out_logprob) {
            // the largest value is kept: z >= 2^43, and both terms have one sign
            const float lnz = log1pf((float)(z - (1ull << kPoint)) * 1.1368683772161603e-13f);
            p.out_logprob[row] = (value - m) / set.tau - lnz;
        }
    };

    Shared* lead = cluster.map_shared_rank(&sh, 0);
    uint32_t lo = kLowest;   // keys below are not kept
    uint32_t hi = ordered(m);
    bool cut_found = false;
    Cut cut = {least, kAll, 0, 0, 0};
    if (set.k || set.top_p < 1.f) {
        uint64_t target = set.k;
        bool by_count = set.k != 0;
        if (by_count) {
            // ---- 2a. a bound for the k-th largest, from the threads' largest
            uint64_t n = 0;
            if (threadIdx.x < kBound)
                for (uint32_t k = 0; k < C; ++k) n += *cluster.map_shared_rank(&sh.bound[kBound - 1 - threadIdx.x], k);
            const uint64_t upto = block_scan(n, sh.scan);
            if (threadIdx.x == 0) sh.words[0] = kLowest;
            __syncthreads();
            if (threadIdx.x < kBound && upto >= set.k && upto - n < set.k) sh.words[0] = bound_edge(kBound - 1 - threadIdx.x);
            __syncthreads();
            lo = (uint32_t)sh.words[0];
        } else {
            // ---- 2b. the sum of all weights, and from it a bound
            Weight s = {0.f, 0.f};
            for (uint32_t v = lane; v < vecs; v += 32) {
                float f[VEC];
                widen(mine[v], f, T());
#pragma unroll
                for (uint32_t i = 0; i < VEC; ++i) add(s, weight_of(f[i]));
            }
            const uint64_t sum = block_scan(fixed(s), sh.scan);
            if (threadIdx.x == kThreads - 1) sh.cta_sum = sum;
            cluster.sync();
            uint64_t z = 0;
            for (uint32_t k = 0; k < C; ++k) z += *cluster.map_shared_rank(&sh.cta_sum, k);
            target = reached_at(set.top_p, z);
            // kept tokens weigh (1 - p) Z / V at least (with room for the roundings here)
            const float w = (1.f - set.top_p) * ((float)z * 1.1368683772161603e-13f) / (float)p.V;
            const float f = m + set.tau * (logf(w) - 0.01f) - fabsf(m) * 1e-6f;
            lo = f > -3e38f ? max(ordered(f + 0.f), kLowest) : kLowest;
            if (lo > hi) lo = hi;
        }
        // ---- 3. all that can be kept in one list?
        if (!by_count || set.k <= kList) {
            for (uint32_t v = lane; v < (vecs + 31) / 32 * 32; v += 32) {
                float f[VEC];
                uint32_t take = 0;
                if (v < vecs) {
                    widen(mine[v], f, T());
#pragma unroll
                    for (uint32_t i = 0; i < VEC; ++i) take |= (ordered(f[i]) >= lo ? 1u : 0u) << i;
                }
                if (!__any_sync(0xFFFFFFFFu, take)) continue;
                const uint32_t n = __popc(take);
                const uint32_t upto = (uint32_t)warp_scan(n), all = __shfl_sync(0xFFFFFFFFu, upto, 31);
                uint32_t at = 0;
                if (lane == 31) at = atomicAdd(&lead->listed, all);
                at = __shfl_sync(0xFFFFFFFFu, at, 31);
                if (at + all > kList) break;  // (counted, so that it is seen)
                at += upto - n;
                while (take) {
                    const uint32_t i = __ffs(take) - 1;
                    take &= take - 1;
                    float value = 0.f;
#pragma unroll
                    for (uint32_t k = 0; k < VEC; ++k) value = k == i ? f[k] : value;
                    lead->list[at++] = (uint64_t)ordered(value) << 32 | (uint32_t)~id_of(v, i);
                }
            }
            cluster.sync();
            const uint32_t n = lead->listed;
            if (n <= kList) {
                // the first CTA does the rest; no one reads the others' memory any more
                if (rank != 0) {
                    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
                    return;
                }
                sort_list(sh.list, n);
                uint64_t w[2], sum = 0;
                for (uint32_t i = 0; i < 2; ++i) {
                    const uint32_t at = 2 * threadIdx.x + i;
                    const uint32_t key = at < n ? (uint32_t)(sh.list[at] >> 32) : 0u;
                    w[i] = at < n && (!set.k || at < set.k) ? fixed(weight_of(unordered(key))) : 0;
                    sum += w[i];
                }
                const uint64_t upto = block_scan(sum, sh.scan);
                if (threadIdx.x == kThreads - 1) sh.words[0] = upto;
                if (threadIdx.x == 0) sh.words[1] = 0;
                __syncthreads();
                if (by_count) target = set.top_p < 1.f ? reached_at(set.top_p, sh.words[0]) : ~0ull;
                uint32_t kept = 0;
                uint64_t below = upto - sum;
                for (uint32_t i = 0; i < 2; ++i) {
                    const uint32_t at = 2 * threadIdx.x + i;
                    const bool keep = at < n && w[i] && below < target && (uint32_t)(sh.list[at] >> 32) >= least;
                    kept += keep;
                    below += w[i];
                }
                kept = (uint32_t)block_scan(kept, sh.scan);
                if (threadIdx.x == kThreads - 1) sh.words[1] = kept;
                __syncthreads();
                kept = (uint32_t)sh.words[1];  // the first so many
                // by id: ~id and the place in the list
                uint64_t order[2];
                for (uint32_t i = 0; i < 2; ++i) {
                    const uint32_t at = 2 * threadIdx.x + i;
                    order[i] = at < kept ? (sh.list[at] & 0xFFFFFFFFull) << 32 | at : 0;
                    sh.weight[at] = w[i];
                }
                for (uint32_t i = 0; i < 2; ++i) {
                    const uint32_t at = 2 * threadIdx.x + i;
                    sh.key[at] = (uint32_t)(sh.list[at] >> 32);
                    sh.list[at] = order[i];
                }
                __syncthreads();
                sort_list(sh.list, kept);
                sum = 0;
                uint32_t at_list[2];
                for (uint32_t i = 0; i < 2; ++i) {
                    const uint32_t at = 2 * threadIdx.x + i;
                    at_list[i] = at < kept ? (uint32_t)sh.list[at] : kAll;
                    w[i] = at < kept ? sh.weight[at_list[i]] : 0;
                    sum += w[i];
                }
                const uint64_t drawn = block_scan(sum, sh.scan);
                if (threadIdx.x == kThreads - 1) sh.words[2] = drawn;
                __syncthreads();
                const uint64_t z = sh.words[2];
                bool exact;
                const uint64_t want = part_of(set.u, z, &exact);
                below = drawn - sum;
                for (uint32_t i = 0; i < 2; ++i) {
                    if (w[i] && below <= want && want < below + w[i])
                        token_is(~(uint32_t)(sh.list[2 * threadIdx.x + i] >> 32), unordered(sh.key[at_list[i]]), z);
                    below += w[i];
                }
                asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
                return;
            }
        }
        // ---- 4. the value at which the target is reached, by histograms over [lo, hi]
        for (int round = 0; round < 2 && !cut_found; ++round) {
            uint64_t above = 0;           // weight of the keys above hi
            uint32_t above_count = 0;
            for (;;) {
                uint32_t shift = 0;
                while ((hi - lo) >> shift >= kBins) ++shift;
                cluster.sync();  // (the tables and the list have been read)
                sh.count[threadIdx.x] = sh.low[threadIdx.x] = sh.high[threadIdx.x] = 0;
                if (threadIdx.x == 0) {
                    sh.listed = 0;
                    sh.found_bin = kAll;
                }
                __syncthreads();
                for (uint32_t v = lane; v < vecs; v += 32) {
                    float f[VEC];
                    widen(mine[v], f, T());
#pragma unroll
                    for (uint32_t i = 0; i < VEC; ++i) {
                        const uint32_t key = ordered(f[i]);
                        if (key < lo || key > hi) continue;
                        const uint32_t bin = (hi - key) >> shift;
                        const uint64_t w = fixed(weight_of(f[i]));
                        atomicAdd(&sh.count[bin], 1);
                        const uint32_t was = atomicAdd(&sh.low[bin], (uint32_t)w);
                        const uint32_t carry = was + (uint32_t)w < was;
                        if ((uint32_t)(w >> 32) + carry) atomicAdd(&sh.high[bin], (uint32_t)(w >> 32) + carry);
                    }
                }
                cluster.sync();
                uint32_t n = 0;
                uint64_t w = 0;
                for (uint32_t k = 0; k < C; ++k) {
                    const Shared* o = cluster.map_shared_rank(&sh, k);
                    n += o->count[threadIdx.x];
                    w += (uint64_t)o->high[threadIdx.x] << 32 | o->low[threadIdx.x];
                }
                const uint64_t upto = block_scan(w, sh.scan), upto_n = block_scan(n, sh.scan);
                const uint64_t have = by_count ? above_count + upto_n : above + upto, step = by_count ? n : w;
                if (have >= target && have - step < target) {
                    sh.found_bin = threadIdx.x;
                    sh.found_count = n;
                    sh.found_before = above + upto - w;
                    sh.found_before_count = above_count + (uint32_t)(upto_n - n);
                    sh.words[3] = w;
                }
                __syncthreads();
                const uint32_t bin = sh.found_bin;
                if (bin == kAll) {  // all of it is kept (k is more than there are)
                    if (by_count && set.top_p < 1.f) {
                        if (threadIdx.x == kThreads - 1) sh.words[2] = above + upto;
                        __syncthreads();
                        cut.above = lo - 1;
                        cut.target = reached_at(set.top_p, sh.words[2]);
                        break;
                    }
                    cut = {max(lo, least), kAll, 0, 0, 0};
                    cut_found = true;
                    break;
                }
                above = sh.found_before;
                above_count = sh.found_before_count;
                const uint32_t in_bin = sh.found_count;
                const uint64_t bin_weight = sh.words[3];
                hi = hi - (bin << shift);
                lo = max(lo, hi - (1u << shift) + 1 > hi ? 0u : hi - (1u << shift) + 1);
                if (in_bin > kList && lo < hi) continue;
                if (in_bin > kList) {
                    // one value: its first `j` ids are kept
                    const uint64_t each = bin_weight / in_bin;
                    uint64_t j = by_count ? target - above_count : (target - above + each - 1) / each;
                    bool again = false;
                    uint64_t next = 0;
                    if (by_count && set.top_p < 1.f) {
                        next = reached_at(set.top_p, above + j * each);
                        if (next <= above) again = true;
                        else if (each) j = min(j, (next - above + each - 1) / each);
                    }
                    if (again) {
                        cut.again = 1;
                        cut.above = hi;
                        cut.target = next;
                    } else {
                        // the j-th of them, counted by warp in the order of the ids
                        uint32_t mine_count = 0;
                        for (uint32_t v = lane; v < vecs; v += 32) {
                            float f[VEC];
                            widen(mine[v], f, T());
#pragma unroll
                            for (uint32_t i = 0; i < VEC; ++i) mine_count += ordered(f[i]) == hi;
                        }
                        mine_count = __reduce_add_sync(0xFFFFFFFFu, mine_count);
                        if (lane == 0) sh.warp_count[warp] = mine_count;
                        cluster.sync();
                        uint64_t before_me = 0;
                        for (uint32_t k = 0; k <= rank; ++k)
                            for (uint32_t q = 0; q < (k < rank ? kWarps : warp); ++q)
                                before_me += *cluster.map_shared_rank(&sh.warp_count[q], k);
                        if (before_me < j && j <= before_me + mine_count) {
                            uint32_t left = (uint32_t)(j - before_me), found = 0;
                            for (uint32_t v0 = 0; v0 < vecs && left; v0 += 32) {
                                const uint32_t v = v0 + lane;
                                uint32_t take = 0;
                                if (v < vecs) {
                                    float f[VEC];
                                    widen(mine[v], f, T());
#pragma unroll
                                    for (uint32_t i = 0; i < VEC; ++i) take |= (ordered(f[i]) == hi ? 1u : 0u) << i;
                                }
                                const uint32_t c = __popc(take), cum = (uint32_t)warp_scan(c);
                                const uint32_t all = __shfl_sync(0xFFFFFFFFu, cum, 31);
                                if (left > all) {
                                    left -= all;
                                    continue;
                                }
                                if (cum >= left && cum - c < left) {
                                    uint32_t skip = left - (cum - c) - 1;
                                    while (skip--) take &= take - 1;
                                    found = id_of(v, __ffs(take) - 1);
                                    for (uint32_t k = 0; k < C; ++k) {
                                        Shared* o = cluster.map_shared_rank(&sh, k);
                                        o->cut.id = found;
                                    }
                                }
                                left = 0;
                            }
                        }
                        cluster.sync();
                        cut = {hi, sh.cut.id, 0, 0, 0};
                    }
                } else {
                    // the bin's tokens, sorted by the first CTA
                    for (uint32_t v = lane; v < vecs; v += 32) {
                        float f[VEC];
                        widen(mine[v], f, T());
#pragma unroll
                        for (uint32_t i = 0; i < VEC; ++i) {
                            const uint32_t key = ordered(f[i]);
                            if (key < lo || key > hi) continue;
                            const uint32_t at = atomicAdd(&lead->listed, 1);
                            if (at < kList) lead->list[at] = (uint64_t)key << 32 | (uint32_t)~id_of(v, i);
                        }
                    }
                    cluster.sync();
                    if (rank == 0) {
                        const uint32_t count = min(in_bin, kList);
                        sort_list(sh.list, count);
                        const uint32_t limit = by_count ? (uint32_t)(target - above_count) : kAll;
                        uint64_t w2[2], sum = 0;
                        for (uint32_t i = 0; i < 2; ++i) {
                            const uint32_t at = 2 * threadIdx.x + i;
                            w2[i] = at < count && at < limit ? fixed(weight_of(unordered((uint32_t)(sh.list[at] >> 32)))) : 0;
                            sum += w2[i];
                        }
                        const uint64_t cum = block_scan(sum, sh.scan);
                        if (threadIdx.x == kThreads - 1) sh.words[0] = cum;
                        __syncthreads();
                        uint64_t reach = target;
                        if (by_count) reach = set.top_p < 1.f ? reached_at(set.top_p, above + sh.words[0]) : ~0ull;
                        uint32_t kept = 0;
                        uint64_t below = above + cum - sum;
                        for (uint32_t i = 0; i < 2; ++i) {
                            const uint32_t at = 2 * threadIdx.x + i;
                            kept += at < count && at < limit && below < reach;
                            below += w2[i];
                        }
                        kept = (uint32_t)block_scan(kept, sh.scan);
                        if (threadIdx.x == kThreads - 1) {
                            Cut c = {kAll, 0, 0, 0, 0};
                            if (kept) {
                                const uint64_t last = sh.list[kept - 1];
                                c.key = (uint32_t)(last >> 32);
                                c.id = ~(uint32_t)last;
                            } else {  // reached among larger values
                                c.again = 1;
                                c.above = hi;
                                c.target = reach;
                            }
                            for (uint32_t k = 0; k < C; ++k) cluster.map_shared_rank(&sh, k)->cut = c;
                        }
                    }
                    cluster.sync();
                    cut = sh.cut;
                }
                if (!cut.again) {
                    cut_found = true;
                    if (least > cut.key) cut = {least, kAll, 0, 0, 0};
                }
                break;
            }
            if (!cut_found) {  // once more, by weight, among the larger values
                by_count = false;
                target = cut.target;
                lo = cut.above + 1;
                hi = ordered(m);
            }
        }
    }

    // ---- 5. the kept weights by warp, in the order of the ids, and the draw
    const auto kept_weight = [&](float f, uint32_t id) -> Weight {
        const uint32_t key = ordered(f);
        if (key < cut.key || (key == cut.key && id > cut.id)) return {0.f, 0.f};
        return weight_of(f);
    };
    Weight s = {0.f, 0.f};
    for (uint32_t v = lane; v < vecs; v += 32) {
        float f[VEC];
        widen(mine[v], f, T());
#pragma unroll
        for (uint32_t i = 0; i < VEC; ++i) add(s, kept_weight(f[i], id_of(v, i)));
    }
    uint64_t sum = warp_scan(fixed(s));
    if (lane == 31) sh.warp_sum[warp] = sum;
    cluster.sync();
    // the warps' sums, each warp for itself: four to a lane
    uint64_t part[kMaxCluster * kWarps / 32], own = 0;
#pragma unroll
    for (uint32_t i = 0; i < kMaxCluster * kWarps / 32; ++i) {
        const uint32_t g = lane * (kMaxCluster * kWarps / 32) + i;
        part[i] = g < C * kWarps ? *cluster.map_shared_rank(&sh.warp_sum[g % kWarps], g / kWarps) : 0;
        own += part[i];
    }
    const uint64_t upto = warp_scan(own), z = __shfl_sync(0xFFFFFFFFu, upto, 31);
    bool exact;
    const uint64_t want = part_of(set.u, z, &exact);
    uint64_t below = upto - own, start = 0;
    uint32_t hit = kAll;
#pragma unroll
    for (uint32_t i = 0; i < kMaxCluster * kWarps / 32; ++i) {
        if (hit == kAll && want < below + part[i] && below <= want) {
            hit = lane * (kMaxCluster * kWarps / 32) + i;
            start = below;
        }
        below += part[i];
    }
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, hit != kAll);
    const int src = who ? __ffs(who) - 1 : 0;
    hit = __shfl_sync(0xFFFFFFFFu, hit, src);
    start = __shfl_sync(0xFFFFFFFFu, start, src);
    if (hit == rank * kWarps + warp) {
        uint64_t left = want - start;
        uint32_t last_id = kAll, got = kAll;  // the last kept: the sums above are rounded another way than those below
        float last_value = 0.f, value = 0.f;
        for (uint32_t v0 = 0; v0 < vecs; v0 += 32) {
            const uint32_t v = v0 + lane;
            float f[VEC];
            uint64_t w[VEC], here = 0;
            if (v < vecs) widen(mine[v], f, T());
#pragma unroll
            for (uint32_t i = 0; i < VEC; ++i) {
                w[i] = v < vecs ? fixed(kept_weight(f[i], id_of(v, i))) : 0;
                here += w[i];
                if (w[i]) {
                    last_id = id_of(v, i);
                    last_value = f[i];
                }
            }
            const uint64_t cum = warp_scan(here), all = __shfl_sync(0xFFFFFFFFu, cum, 31);
            if (left >= all) {
                left -= all;
                continue;
            }
            uint64_t b = cum - here;
            if (left >= b && left < cum) {
#pragma unroll
                for (uint32_t i = 0; i < VEC; ++i) {
                    if (w[i] && got == kAll && left < b + w[i]) {
                        got = id_of(v, i);
                        value = f[i];
                    }
                    b += w[i];
                }
            }
            break;
        }
        const uint32_t found = __ballot_sync(0xFFFFFFFFu, got != kAll);
        if (found) {
            if (got != kAll) token_is(got, value, z);
        } else {
            const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, last_id + 1);  // (none: 0)
            if (last_id != kAll && last_id + 1 == most) token_is(last_id, last_value, z);
        }
    }
    cluster.sync();  // (the sums have been read)
}

static_assert((kMaxSlice + kThreads * 4) * 4 + sizeof(Shared) <= 227 * 1024, "the longest rows fit");

template <typename T>
lp_status launch_sample(SampleParams p, lp_stream_t stream) {
    constexpr uint32_t kVec = Vec<T>::kElems, kUnit = kWarps * 32 * kVec;  // elements of whole rounds of a CTA
    static std::atomic<uint64_t> smem_set;
    // CTAs of a row: slices of 16384 elements at most (the smallest number that gives them), eight at most
    const uint64_t n = (uint64_t)p.V + kVec - 1;
    uint32_t c = 1;
    while (c < kMaxCluster && n > (uint64_t)c * 16384) c *= 2;
    const uint32_t rounds = (uint32_t)((n + (uint64_t)c * kUnit - 1) / ((uint64_t)c * kUnit));
    p.chunk = rounds * 32 * kVec;
    auto kernel = k_sample<T>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), kMaxSlice * sizeof(T) + kUnit * sizeof(T), &smem_set)) return LP_ERR_CUDA;
    return launch(kernel, dim3(p.T * c), kThreads, (size_t)p.chunk * kWarps * sizeof(T), stream, c, p);
}

}  // namespace

extern "C" lp_status lp_head_sample(const void* logits, uint32_t dtype, uint32_t T, uint32_t V, uint64_t stride,
                                    const float* uniform, const uint32_t* row_offsets, uint32_t B,
                                    const float* temperature, const int32_t* top_k, const float* top_p,
                                    const float* min_p, uint32_t* out, float* out_logprob, void* workspace,
                                    size_t workspace_bytes, lp_stream_t stream) {
    if (T == 0 || V == 0) return LP_ERR_SHAPE;
    if (!logits || !uniform || !out) return LP_ERR_NULL;
    if (dtype != LP_F32 && dtype != LP_BF16 && dtype != LP_F16) return LP_ERR_DTYPE;
    if (V > LP_MAX_SAMPLE_VOCAB || stride < V || T > 0x7FFFFFFFu / kMaxCluster || B == 0 || (!row_offsets && B != T))
        return LP_ERR_SHAPE;
    if (!aligned_to(logits, dtype_bytes(dtype)) || !aligned_to(uniform, 4) || !aligned_to(row_offsets, 4) ||
        !aligned_to(temperature, 4) || !aligned_to(top_k, 4) || !aligned_to(top_p, 4) || !aligned_to(min_p, 4) ||
        !aligned_to(out, 4) || !aligned_to(out_logprob, 4))
        return LP_ERR_SHAPE;
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < kHeaderBytes) return LP_ERR_WORKSPACE;
    SampleParams p = {};
    p.logits = logits;
    p.uniform = uniform;
    p.row_offsets = row_offsets;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.out = out;
    p.out_logprob = out_logprob;
    p.status = static_cast<uint32_t*>(workspace);
    p.stride = stride;
    p.T = T;
    p.V = V;
    p.B = B;
    if (dtype == LP_F32) return launch_sample<float>(p, stream);
    if (dtype == LP_BF16) return launch_sample<__nv_bfloat16>(p, stream);
    return launch_sample<__half>(p, stream);
}
