// Draw of the next token (include/lp_head.h): temperature, top-k, top-p and min-p, from a given
// random number a row.
//
// A row belongs to a cluster of up to eight CTAs, each with a slice of it in shared memory, read
// from HBM once. Weights exp((x - max) / tau) are formed with about 34 correct bits (a table of 256
// powers, and a short series for what is left of the exponent) and added as pairs of f32 or as
// integers of 2^-43: the token is a comparison of sums of up to some hundred thousand weights with
// each other, and f32's rounding would move it in a few rows of a hundred. All three filters keep a
// prefix of the order (value descending, id ascending), so that what is kept is told by the last
// kept (value, id):
//   top-k: each CTA tells a value that enough of its threads' largest reach (a coarse histogram);
//          what lies above the least of these is listed and ranked by the cluster's first CTA.
//   top-p: what weighs less than (1 - p) Z / V is never kept. Where Z is small the rest is listed
//          as well. Else, or if it does not fit, a histogram over the values' bits with rounded
//          weights finds the bins in which p Z can be reached; what lies above them is summed
//          exactly, what lies in them is listed. Bins of more than fits are cut again; a single
//          value is cut by id.
// The draw follows the ids: the kept weights are summed by warp, and the CTA in which u Z falls
// walks that warp's part once more. CTAs write what the others need into their shared memory
// before a barrier of the cluster.
#include <cooperative_groups.h>

#include <type_traits>

#include "lp_head_common.h"

namespace {

using namespace lph;
namespace cg = cooperative_groups;

constexpr uint32_t kThreads = 384, kWarps = kThreads / 32;
constexpr uint32_t kResident = 3;  // CTAs per SM, with slices of up to 16384 f32
constexpr uint32_t kMaxCluster = 8;
constexpr uint32_t kList = kThreads;  // tokens that are ranked
constexpr uint32_t kBins = 2 * kThreads;
constexpr uint32_t kBound = 256;
constexpr uint32_t kTable = 256;
constexpr uint32_t kLowest = 0x00800000u;  // ordered() of the lowest finite value
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kUnit = 8796093022208.f;  // 2^43: weights as integers, the largest one is about that
constexpr float kFewWeights = 8.f;   // Z up to which a top-p row's tokens are listed at once
// Rounded weights of a histogram: all of them make 2^30; what the roundings can add up to.
constexpr uint32_t kWhole = 1u << 30, kMargin = 1u << 18;
static_assert(LP_MAX_SAMPLE_VOCAB / 2 + (kWhole >> 16) < kMargin, "half a unit a token, and the weights' f32 errors");

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
    uint32_t chunk;  // elements of a warp: whole vectors
};

// A value's bits in the order of the values (both zeros were made one before).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
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
    float top_p, min_p, u;
    uint32_t k;            // 0: off
};

struct Cut {
    uint32_t key, id;      // kept: a larger key, or this one with an id up to this
    uint32_t again;        // the search goes on among keys above `above`, for the weight `target` of `total`
    uint32_t above;
    uint64_t target, total;
};

struct Told {              // by each CTA
    uint32_t top;          // ordered() of its largest value (a NaN's is above all)
    uint32_t share, whole; // keys that ceil(k / CTAs), and k, of its threads' largest reach
};

struct Range {             // keys among which the cut is
    uint32_t lo, hi;
    uint32_t end;          // the least key of the first bin
    uint32_t in;           // how many they hold
    uint32_t above_count;  // how many lie above them, in the histogram's range
    uint32_t none;         // by count: there are not as many
    uint32_t narrowed, more;  // than before; than one bin
    float grow;            // what the rounded weights may be multiplied with
};

struct Draw {              // where the token is
    uint64_t start, z;     // the kept weights before the warp that has it, and all
    uint32_t warp;
};

struct Shared {
    union {
        uint64_t list[kList];    // key << 32 | ~id; the ranked tokens' weights
        uint32_t bound[kBound];  // (before the list)
    };
    union {
        struct {
            uint32_t weight[kBins], count[kBins];
        };
        uint64_t stage[kList];   // a CTA's part of the list; the ranked list
    };
    float2 table[kTable];
    uint64_t scan[kWarps];
    uint64_t warp_sum[kMaxCluster * kWarps];
    Told told[kMaxCluster];
    Setting set;
    Cut cut;
    Draw draw;
    Range range;
    uint32_t listed, staged, place, top;
    uint32_t first_bin, last_bin, in_bins, in_weight, above_bins;
};

// 2^(j / 256) as pairs of f32, at compile time, by the exponential's series.
struct Table {
    float2 at[kTable];
};
constexpr Table make_table() {
    Table t = {};
    for (uint32_t j = 0; j < kTable; ++j) {
        const double y = 0.6931471805599453094 * j / kTable;
        double sum = 1.0;
        for (int n = 24; n > 0; --n) sum = 1.0 + sum * y / n;
        t.at[j].x = (float)sum;
        t.at[j].y = (float)(sum - (double)(float)sum);
    }
    return t;
}
__device__ const Table g_table = make_table();

struct Scale {             // of a row
    float m, low;          // largest value; values below `low` weigh 0
    float base, chi, clo;  // exponents are (x - base) (chi + clo) - shift
    float magic;           // 1.5 * 2^15, of which an ulp is 2^-8, less the shift: a multiple of 2^-8
};
__device__ __forceinline__ Scale scale_of(float m, const Setting& s) {
    // where exp falls below 2^-40 (or f32 ends)
    const float low = fmaxf(fmaxf(m - 27.725887f * s.tau, m - 3e38f), -3.402823466e38f);
    // Far out the largest value is subtracted first: exact there, since what weighs more than
    // 2^-40 is within a factor of two of it.
    const bool far = !(fabsf(m) * s.chi < 8192.f);
    const float shift = far ? 0.f : (m * s.chi + 49152.f) - 49152.f;
    return {m, low, far ? m : 0.f, s.chi, s.clo, 49152.f - shift};
}

struct Weight {
    float hi, lo;  // hi + lo, |lo| <= 2^-8 hi
};
// exp((x - m) / tau) times a factor between 2^(-1/512) and 2^(1/512) that is the row's; 0 below
// 2^-40. About 20 operations of f32.
__device__ __forceinline__ Weight weigh(float x, const Scale& r, const float2* table) {
    const float y = fmaxf(x, r.low) - r.base;
    const float t = fmaf(y, r.chi, r.magic), grid = t - r.magic;  // of 2^-8, exact
    const float g = fmaf(y, r.clo, fmaf(y, r.chi, -grid));        // |g| <= 2^-9
    const float q = g * fmaf(g, fmaf(g, 0.0555041087f, 0.240226507f), 0.693147181f);  // 2^g - 1
    const uint32_t bits = __float_as_uint(t);  // 0x47400000 + the exponent in units of 2^-8
    const float2 e = table[bits & (kTable - 1)];
    const uint32_t power = ((bits << 15) & 0xFF800000u) + ((127u - 0x474000u) << 23);
    const float scale = x >= r.low ? __uint_as_float(power) : 0.f;
    return {e.x * scale, fmaf(e.x, q, e.y) * scale};
}
__device__ __forceinline__ uint64_t fixed(Weight w) { return __float2ull_rn(w.hi * kUnit) + (uint64_t)__float2ll_rn(w.lo * kUnit); }
// Sums of weights, as pairs.
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

template <typename N>
__device__ __forceinline__ N warp_scan(N v) {  // inclusive
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
        const N o = __shfl_up_sync(0xFFFFFFFFu, v, k);
        if (lane >= k) v += o;
    }
    return v;
}
// Inclusive scan over the CTA's threads, and the sum of all.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* scratch, uint64_t* all) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_scan(v);
    __syncthreads();
    if (lane == 31) scratch[warp] = v;
    __syncthreads();
    uint64_t before = 0, sum = 0;
#pragma unroll
    for (uint32_t k = 0; k < kWarps; ++k) {
        before += k < warp ? scratch[k] : 0;
        sum += scratch[k];
    }
    *all = sum;
    return v + before;
}

// Threads that share a key of a list of n, as a power of two, so that n keys keep the CTA busy.
__device__ __forceinline__ uint32_t sharing(uint32_t n) { return n <= kList / 8 ? 3 : n <= kList / 4 ? 2 : n <= kList / 2 ? 1 : 0; }
// n different keys (n <= kList) of `from` in descending order, to `to`, each ranked by counting the
// larger ones (200 of them: 1 us; a bitonic sort waits for the CTA at each of 36 steps).
__device__ __forceinline__ void sort_list(const uint64_t* from, uint64_t* to, uint32_t n) {
    const uint32_t t = threadIdx.x, shift = sharing(n), at = t >> shift, parts = 1u << shift;
    const uint64_t key = at < n ? from[at] : 0;
    uint32_t rank = 0;
#pragma unroll 8
    for (uint32_t j = t & (parts - 1); j < n; j += parts) rank += from[j] > key;
    for (uint32_t k = 1; k < parts; k *= 2) rank += __shfl_xor_sync(0xFFFFFFFFu, rank, k);
    if (at < n && (t & (parts - 1)) == 0) to[rank] = key;
    __syncthreads();
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

__device__ __forceinline__ Setting setting_of(const SampleParams& p, uint32_t row, bool report) {
    Setting s = {};
    // (those of request `row`, which it is where every request has one row, are asked for at once)
    int b = (int)min(row, p.B - 1);
    float tau = p.temperature ? p.temperature[b] : 1.f, top_p = p.top_p ? p.top_p[b] : 1.f, min_p = p.min_p ? p.min_p[b] : 0.f;
    int k = p.top_k ? p.top_k[b] : 0;
    const float u = p.uniform[row];
    const int found = request_of(p.row_offsets, p.B, row);
    if (found < 0) {
        if (report) flag(p.status, LP_ERR_OFFSETS);
        return s;
    }
    if (found != b) {
        b = found;
        tau = p.temperature ? p.temperature[b] : 1.f;
        top_p = p.top_p ? p.top_p[b] : 1.f;
        min_p = p.min_p ? p.min_p[b] : 0.f;
        k = p.top_k ? p.top_k[b] : 0;
    }
    s.ok = 1;
    if (!(tau >= 0.f && tau <= 3.402823466e38f)) {
        s.ok = 0;
        if (report) flag(p.status, LP_ERR_TEMPERATURE);
    }
    if (!(top_p >= 0.f && top_p <= 1.f) || !(min_p >= 0.f && min_p <= 1.f) || !(u >= 0.f && u < 1.f)) {
        s.ok = 0;
        if (report) flag(p.status, LP_ERR_SAMPLING);
    }
    s.k = k > 0 && (uint32_t)k < p.V ? (uint32_t)k : 0;
    if (tau == 0.f) {
        tau = 1.f;
        s.k = 1;
    }
    // log2(e) = 1.44269502 + 1.92596299e-8 over tau, as a pair: the quotient and its remainder's
    tau = fminf(fmaxf(tau, 7.8886091e-31f), 1.2676506e30f);  // 2^-100, 2^100
    s.tau = tau;
    s.chi = 1.44269502f / tau;
    s.clo = (fmaf(-s.chi, tau, 1.44269502f) + 1.92596299e-8f) / tau;
    s.top_p = top_p;
    s.min_p = min_p;
    s.u = u;
    return s;
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kResident) k_sample(const SampleParams p) {
    constexpr uint32_t VEC = Vec<T>::kElems;
    constexpr float kInf = __builtin_huge_valf();
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ Shared sh;
    uint4* slice = reinterpret_cast<uint4*>(smem_raw);
    const cg::cluster_group cluster = cg::this_cluster();
    const uint32_t C = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t row = blockIdx.x / C, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    pdl_trigger();
    const float2 power = t < kTable ? g_table.at[t] : make_float2(0.f, 0.f);
    if (t < kBound) sh.bound[t] = 0;
    if (t == 0) sh.staged = sh.listed = sh.top = 0;
    __syncthreads();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (waited for before others' memory is written to)
    pdl_wait();

    // The row in units of aligned vectors: element i of the row is number i + before. Slices and the
    // warps' parts of them are whole vectors; what lies outside the row becomes -inf.
    const T* x = static_cast<const T*>(p.logits) + (uint64_t)row * p.stride;
    const uint32_t before = (uint32_t)(reinterpret_cast<uintptr_t>(x) / sizeof(T)) % VEC;
    const uint32_t vecs = p.chunk / VEC;                     // of a warp
    const uint32_t begin = (rank * kWarps + warp) * p.chunk; // number of the warp's first element
    uint4* mine = slice + warp * vecs;
    const T* values = reinterpret_cast<const T*>(mine);
    const auto id_of = [&](uint32_t element) { return begin + element - before; };  // of the warp's part

    // ---- 1. read; the largest value, and threads' largest in coarse bins; the setting, by one thread
    float top = -kInf;
#pragma unroll 8
    for (uint32_t v = lane; v < vecs; v += 32) {
        const uint32_t at = begin + v * VEC;
        uint4 w;
        if (at >= before && at + VEC <= p.V + before) {
            w = *reinterpret_cast<const uint4*>(x + (at - before));
        } else {
            T e[VEC];
#pragma unroll
            for (uint32_t i = 0; i < VEC; ++i) {
                const uint32_t n = at + i;
                e[i] = n >= before && n < p.V + before ? x[n - before] : from_f32<T>(-kInf);
            }
            memcpy(&w, e, 16);
        }
        mine[v] = w;
        float f[VEC];
        widen(w, f, T());
#pragma unroll
        for (uint32_t i = 0; i < VEC; i += 2) top = max_nan(top, f[i], f[i + 1]);
    }
    if (t == kThreads - 1) sh.set = setting_of(p, row, rank == 0);
    __syncwarp();
    if (t < kTable) sh.table[t] = power;
    if (top > -kInf) atomicAdd(&sh.bound[bound_bin(top)], 1);
    const uint32_t warp_top = __reduce_max_sync(0xFFFFFFFFu, ordered(top));  // (max.NaN's NaN is positive)
    if (lane == 0) atomicMax(&sh.top, warp_top);
    __syncthreads();
    const Setting set = sh.set;
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 0) {
        Told told = {sh.top, kLowest, kLowest};
        if (set.k) {
            // from the top: lane 0 has the largest bins
            uint32_t n[kBound / 32], sum = 0;
#pragma unroll
            for (uint32_t i = 0; i < kBound / 32; ++i) sum += n[i] = sh.bound[kBound - 1 - (lane * (kBound / 32) + i)];
            const uint32_t upto = warp_scan(sum), share = (set.k + C - 1) / C;
            uint32_t have = upto - sum, s = kAll, w = kAll;
#pragma unroll
            for (uint32_t i = 0; i < kBound / 32; ++i) {
                const uint32_t bin = kBound - 1 - (lane * (kBound / 32) + i);
                if (have < share && have + n[i] >= share) s = bin;
                if (have < set.k && have + n[i] >= set.k) w = bin;
                have += n[i];
            }
            s = __reduce_min_sync(0xFFFFFFFFu, s);
            w = __reduce_min_sync(0xFFFFFFFFu, w);
            told.share = s == kAll ? kLowest : bound_edge(s);
            told.whole = w == kAll ? kLowest : bound_edge(w);
        }
        if (lane < C) cluster.map_shared_rank(&sh, lane)->told[rank] = told;
    }
    cluster.sync();
    const Told told = lane < C ? sh.told[lane] : Told{0, kAll, 0};
    uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, told.top);
    uint32_t lo = max(__reduce_min_sync(0xFFFFFFFFu, told.share), __reduce_max_sync(0xFFFFFFFFu, told.whole));  // keys below are not kept
    if (!set.ok || hi < kLowest || hi >= ordered(kInf)) {
        if (rank == 0 && t == 0) {
            if (set.ok) flag(p.status, LP_ERR_LOGITS);
            p.out[row] = kAll;
            if (p.out_logprob) p.out_logprob[row] = __uint_as_float(0x7FC00000u);
        }
        return;
    }
    const float m = unordered(hi);
    const Scale scale = scale_of(m, set);
    const auto weight_of = [&](float f) { return weigh(f, scale, sh.table); };
    const Weight most = weight_of(m);
    // min-p: what weighs less than that is not kept. `least` is a key below all that are (room for
    // the roundings here), the weights decide.
    uint32_t least = kLowest;
    if (set.min_p > 0.f) {
        const float f = m + set.tau * (__logf(set.min_p) - 0.01f) - fabsf(m) * 1e-6f;
        least = f > -3e38f ? min(max(ordered(f + 0.f), kLowest), hi) : kLowest;
    }
    const auto enough = [&](Weight w) {
        return set.min_p == 0.f || (double)w.hi + (double)w.lo >= (double)set.min_p * ((double)most.hi + (double)most.lo);
    };
    const auto token_is = [&](uint32_t id, float value, uint64_t z) {
        p.out[row] = id;
        if (p.out_logprob) {
            // both terms have one sign: the largest value is kept
            const uint64_t one = fixed(most);
            const float lnz = z > one ? log1pf((float)(z - one) / (float)one) : 0.f;
            p.out_logprob[row] = (value - m) / set.tau - lnz;
        }
    };
    // Visits the warp's elements with values in [from, to], two at a time: body(element, element or
    // kAll, value, value). Lanes take them out of masks of 32, so that few cost little.
    const auto visit = [&](float from, float to, auto body) {
        for (uint32_t v0 = 0; v0 < vecs; v0 += 32 * (32 / VEC)) {
            uint32_t take = 0;
#pragma unroll
            for (uint32_t j = 0; j < 32 / VEC; ++j) {
                const uint32_t v = v0 + j * 32 + lane;
                if (v < vecs) {
                    float f[VEC];
                    widen(mine[v], f, T());
                    float high = f[0];
#pragma unroll
                    for (uint32_t i = 1; i < VEC; ++i) high = fmaxf(high, f[i]);
                    if (!__any_sync(__activemask(), high >= from)) continue;
#pragma unroll
                    for (uint32_t i = 0; i < VEC; ++i)
                        if (f[i] >= from && f[i] <= to) take |= 1u << (j * VEC + i);
                }
            }
            const auto next = [&] {
                if (!take) return kAll;
                const uint32_t b = __ffs(take) - 1;
                take &= take - 1;
                return (v0 + b / VEC * 32 + lane) * VEC + b % VEC;
            };
            while (__any_sync(0xFFFFFFFFu, take)) {
                const uint32_t e0 = next(), e1 = next();
                const float f0 = e0 == kAll ? -kInf : to_f32(values[e0]) + 0.f, f1 = e1 == kAll ? -kInf : to_f32(values[e1]) + 0.f;
                body(e0, e1, f0, f1);
            }
        }
    };
    const auto warp_total = [&](uint64_t v) {
#pragma unroll
        for (int k = 16; k > 0; k /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, k);
        return v;
    };
    // All weights of the warp's elements.
    const auto add_all = [&](Weight& s) {
#pragma unroll 1
        for (uint32_t v = lane; v < vecs; v += 32) {
            float f[VEC];
            widen(mine[v], f, T());
            float high = f[0];
#pragma unroll
            for (uint32_t i = 1; i < VEC; ++i) high = fmaxf(high, f[i]);
            if (!__any_sync(__activemask(), high >= scale.low)) continue;
#pragma unroll
            for (uint32_t i = 0; i < VEC; ++i) add(s, weight_of(f[i]));
        }
    };
    // The warp's sum, told to all.
    const auto tell_warp = [&](uint64_t sum) {
        if (lane < C) cluster.map_shared_rank(&sh, lane)->warp_sum[rank * kWarps + warp] = sum;
    };
    const auto told_total = [&] {  // of what all warps told
        uint64_t sum = 0;
#pragma unroll
        for (uint32_t i = 0; i < kMaxCluster * kWarps; i += 32) sum += i + lane < C * kWarps ? sh.warp_sum[i + lane] : 0;
        return warp_total(sum);
    };
    // The sum over all threads of the cluster.
    const auto cluster_total = [&](uint64_t v) {
        tell_warp(warp_total(v));
        cluster.sync();
        return told_total();
    };
    // Where u Z falls among the warps' sums; by a whole warp.
    const auto draw_warp = [&] {
        constexpr uint32_t kEach = kMaxCluster * kWarps / 32;  // of the warps' sums to a lane
        uint64_t part[kEach], own = 0;
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) {
            const uint32_t g = lane * kEach + i;
            part[i] = g < C * kWarps ? sh.warp_sum[g] : 0;
            own += part[i];
        }
        const uint64_t upto = warp_scan(own);
        Draw d = {0, __shfl_sync(0xFFFFFFFFu, upto, 31), kAll};
        bool exact;
        const uint64_t want = part_of(set.u, d.z, &exact);
        uint64_t below = upto - own;
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i) {
            if (below <= want && want < below + part[i]) {
                d.warp = lane * kEach + i;
                d.start = below;
            }
            below += part[i];
        }
        const int src = __ffs(__ballot_sync(0xFFFFFFFFu, d.warp != kAll)) - 1;  // (one lane: want < z)
        d.warp = __shfl_sync(0xFFFFFFFFu, d.warp, src);
        d.start = __shfl_sync(0xFFFFFFFFu, d.start, src);
        return d;
    };

    Shared* lead = cluster.map_shared_rank(&sh, 0);
    // Tokens into the CTA's part of the list, and the parts into the first CTA's, which ends with a barrier of
    // the cluster.
    const auto stage = [&](uint32_t e0, uint32_t e1, float f0, float f1) {
        const auto one = [&](uint32_t e, float f) {
            const uint32_t take = __ballot_sync(0xFFFFFFFFu, e != kAll);
            if (!take) return;
            uint32_t at = 0;
            if (lane == 0) at = atomicAdd(&sh.staged, __popc(take));
            at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(take & ((1u << lane) - 1));
            if (e != kAll && at < kList) sh.stage[at] = (uint64_t)ordered(f) << 32 | (uint32_t)~id_of(e);
        };
        one(e0, f0);
        one(e1, f1);
    };
    const auto send_list = [&] {
        __syncthreads();
        const uint32_t n = sh.staged;
        if (t == 0) sh.place = n ? atomicAdd(&lead->listed, n) : 0u;
        __syncthreads();
        const uint32_t place = sh.place;
        if (place <= kList && n <= kList - place)
            for (uint32_t i = t; i < n; i += kThreads) lead->list[place + i] = sh.stage[i];
        cluster.sync();
    };

    Cut cut = {least, kAll, 0, 0, 0, 0};
    bool drawn = false;  // the first CTA has told where the token is
    if (set.k || set.top_p < 1.f) {
        uint64_t target = set.k;
        bool by_count = set.k != 0, few = set.k <= kList;
        float unit = 1.f;  // of the rounded weights: weights times that
        if (!by_count) {
            // ---- 2. the sum of all weights, and from it a bound
            Weight s = {0.f, 0.f};
            add_all(s);
            const uint64_t z = cluster_total(fixed(s));
            target = reached_at(set.top_p, z);
            const float sum = (float)z / kUnit;
            unit = (float)kWhole / sum;
            // kept tokens weigh (1 - p) Z / V at least (with room for the roundings here)
            const float f = m + set.tau * (__logf((1.f - set.top_p) * sum / (float)p.V) - 0.02f) - fabsf(m) * 1e-6f;
            lo = f > -3e38f ? min(max(ordered(f + 0.f), kLowest), hi) : kLowest;
            few = sum < kFewWeights;
        }
        // ---- 3. all that can be kept in one list?
        if (few) {
            visit(unordered(lo), m, stage);
            send_list();
            const uint32_t n = lead->listed;
            if (n <= kList) {
                // the first CTA does the rest; the others have read its count, and no one reads theirs
                if (rank != 0) {
                    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
                    return;
                }
                sort_list(sh.list, sh.stage, n);
                const uint64_t ranked = t < n ? sh.stage[t] : 0;
                const bool counts = t < n && (!set.k || t < set.k);
                const Weight weight = weight_of(counts ? unordered((uint32_t)(ranked >> 32)) : -kInf);
                const uint64_t w = fixed(weight);
                uint64_t all, kept;
                const uint64_t below = block_scan(w, sh.scan, &all) - w;
                if (by_count) target = set.top_p < 1.f ? reached_at(set.top_p, all) : ~0ull;
                if (t < n) sh.list[t] = w;  // (the list is in `stage` now)
                (void)block_scan(w && enough(weight) && below < target, sh.scan, &kept);
                // The first `kept` of them, in the order of their ids: what lies below each.
                const uint32_t n_kept = (uint32_t)kept, shift = sharing(n_kept), at = t >> shift, parts = 1u << shift;
                const uint64_t entry = at < n_kept ? sh.stage[at] : 0;
                const uint32_t not_id = (uint32_t)entry;
                uint64_t under = 0, z = 0;
#pragma unroll 8
                for (uint32_t j = t & (parts - 1); j < n_kept; j += parts) {
                    const uint64_t wj = sh.list[j];
                    under += (uint32_t)sh.stage[j] > not_id ? wj : 0;
                    z += wj;
                }
                for (uint32_t k = 1; k < parts; k *= 2) {
                    under += __shfl_xor_sync(0xFFFFFFFFu, under, k);
                    z += __shfl_xor_sync(0xFFFFFFFFu, z, k);
                }
                bool exact;
                const uint64_t want = part_of(set.u, z, &exact);
                if (at < n_kept && (t & (parts - 1)) == 0 && under <= want && want < under + sh.list[at])
                    token_is(~not_id, unordered((uint32_t)(entry >> 32)), z);
                asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
                return;
            }
        }
        // ---- 4. the value at which the target is reached, by histograms over [lo, hi]
        bool found = false, read = few;  // whether others may still read the tables and the list
        uint64_t above = 0;              // weight of the keys above hi, and (by count) their number
        uint32_t above_count = 0;
        for (int n_hist = 0; n_hist < 64 && !found; ++n_hist) {  // (a bound only: each cuts the range)
            uint32_t shift = 0;
            while ((hi - lo) >> shift >= kBins) ++shift;
            if (read) cluster.sync();
            read = true;
            for (uint32_t i = t; i < kBins; i += kThreads) sh.weight[i] = sh.count[i] = 0;
            if (t == 0) {
                sh.listed = sh.staged = sh.in_bins = sh.in_weight = 0;
                sh.first_bin = sh.last_bin = kAll;
            }
            __syncthreads();
            {
                const float from = unordered(lo), to = unordered(hi), chi = scale.chi, log_unit = scale.magic - 49152.f + __log2f(unit);
                const auto fill = [&](auto weighted) {
#pragma unroll 1
                    for (uint32_t v = lane; v < vecs; v += 32) {
                        float f[VEC];
                        widen(mine[v], f, T());
#pragma unroll
                        for (uint32_t i = 0; i < VEC; ++i) {
                            if (!(f[i] >= from && f[i] <= to)) continue;
                            const uint32_t bin = (hi - ordered(f[i])) >> shift;
                            atomicAdd(&sh.count[bin], 1);
                            if constexpr (decltype(weighted)::value) {
                                float w;
                                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(fmaf(f[i] - scale.base, chi, log_unit)));
                                atomicAdd(&sh.weight[bin], __float2uint_rn(w));
                            }
                        }
                    }
                };
                if (by_count) fill(std::false_type()); else fill(std::true_type());
            }
            cluster.sync();
            // The first CTA adds the tables up and finds the bins in which the target can be reached.
            if (rank == 0) {
                constexpr uint32_t kEach = kBins / kThreads;
                uint32_t n[kEach] = {}, w[kEach] = {}, n_all = 0, w_all = 0;
                for (uint32_t k = 0; k < C; ++k) {
                    const Shared* o = cluster.map_shared_rank(&sh, k);
#pragma unroll
                    for (uint32_t i = 0; i < kEach; ++i) {
                        n[i] += o->count[kEach * t + i];
                        w[i] += o->weight[kEach * t + i];
                    }
                }
#pragma unroll
                for (uint32_t i = 0; i < kEach; ++i) {
                    n_all += n[i];
                    w_all += w[i];
                }
                uint64_t all;
                const uint64_t upto = block_scan((uint64_t)n_all << 32 | w_all, sh.scan, &all);  // (neither passes 32 bits)
                const uint32_t n_before = (uint32_t)(upto >> 32) - n_all, w_before = (uint32_t)upto - w_all;
                const uint32_t aim = by_count ? (uint32_t)target - above_count
                                              : (uint32_t)((target > above ? (float)(target - above) : 0.f) / kUnit * unit);
                const uint32_t slack = by_count ? 0 : kMargin, from = max(aim, slack + 1) - slack, to = aim + slack;
                uint32_t have = by_count ? n_before : w_before;
#pragma unroll
                for (uint32_t i = 0; i < kEach; ++i) {
                    const uint32_t next = have + (by_count ? n[i] : w[i]);
                    if (have < from && next >= from) sh.first_bin = kEach * t + i;
                    if (have < to && next >= to) sh.last_bin = kEach * t + i;
                    have = next;
                }
                __syncthreads();
                const uint32_t bins = (hi - lo) >> shift, last = min(sh.last_bin, bins), first = min(sh.first_bin, last);
                uint32_t in_n = 0, in_w = 0, below = n_before;
#pragma unroll
                for (uint32_t i = 0; i < kEach; ++i) {
                    const uint32_t bin = kEach * t + i;
                    if (bin == first) sh.above_bins = below;
                    in_n += bin >= first && bin <= last ? n[i] : 0;
                    in_w += bin >= first && bin <= last ? w[i] : 0;
                    below += n[i];
                }
                if (in_n) atomicAdd(&sh.in_bins, in_n);
                if (in_w) atomicAdd(&sh.in_weight, in_w);
                __syncthreads();
                if (t < C) {
                    Range r;
                    r.lo = last == bins ? lo : hi - (((last + 1) << shift) - 1);
                    r.hi = hi - (first << shift);
                    r.end = hi - (((first + 1) << shift) - 1);
                    r.in = sh.in_bins;
                    r.above_count = sh.above_bins;
                    r.none = by_count && sh.first_bin == kAll;
                    r.narrowed = first != 0 || last != bins;
                    r.more = first != last;
                    r.grow = (float)kWhole / ((float)sh.in_weight + 2.f * (float)kMargin);
                    cluster.map_shared_rank(&sh, t)->range = r;
                }
            }
            cluster.sync();  // (the tables have been read, too: the list takes their place)
            const Range range = sh.range;
            if (range.none) {  // all of it is kept
                if (set.top_p == 1.f) {
                    cut = {max(lo, least), kAll, 0, 0, 0, 0};
                    found = true;
                    break;
                }
                Weight s = {0.f, 0.f};
                add_all(s);
                const uint64_t z = cluster_total(fixed(s));
                by_count = false;
                target = reached_at(set.top_p, z);
                unit = (float)kWhole * kUnit / (float)z;
                continue;
            }
            above_count += range.above_count;
            lo = range.lo;
            hi = range.hi;
            // the weights above them, exactly, by warp; what lies in them is listed, where it fits
            const bool fits = range.in <= kList;
            {
                Weight s = {0.f, 0.f};
                const float to = unordered(hi);
                visit(fits ? unordered(lo) : to, m, [&](uint32_t e0, uint32_t e1, float f0, float f1) {
                    add(s, weight_of(f0 > to ? f0 : -kInf));
                    add(s, weight_of(f1 > to ? f1 : -kInf));
                    if (fits) stage(f0 > to ? kAll : e0, f1 > to ? kAll : e1, f0, f1);
                });
                tell_warp(warp_total(fixed(s)));
            }
            if (fits) send_list(); else cluster.sync();
            above = told_total();
            if (fits) {
                // ranked by the first CTA
                if (rank == 0) {
                    sort_list(sh.list, sh.stage, range.in);
                    const uint32_t limit = by_count ? min(range.in, (uint32_t)target - above_count) : range.in;
                    const uint64_t ranked = t < limit ? sh.stage[t] : 0;
                    const uint32_t key = (uint32_t)(ranked >> 32), id = ~(uint32_t)ranked;
                    const uint64_t w = fixed(weight_of(t < limit ? unordered(key) : -kInf));
                    uint64_t sum, kept;
                    const uint64_t below = above + block_scan(w, sh.scan, &sum) - w;
                    uint64_t goal = target;
                    if (by_count) goal = set.top_p < 1.f ? reached_at(set.top_p, above + sum) : ~0ull;
                    const bool keep = t < limit && below < goal;
                    (void)block_scan(keep, sh.scan, &kept);
                    Cut c = {kAll, 0, 1, hi, goal, above + sum};  // reached among larger values
                    Draw d = {};
                    if (kept) {
                        const uint64_t last = sh.stage[kept - 1];
                        c = {(uint32_t)(last >> 32), ~(uint32_t)last, 0, 0, 0, 0};
                        if (set.min_p == 0.f) {  // the warps' sums are complete with these
                            if (keep && w)
                                atomicAdd(reinterpret_cast<unsigned long long*>(&sh.warp_sum[(id + before) / p.chunk]), (unsigned long long)w);
                            __syncthreads();
                            d = draw_warp();
                        }
                    }
                    if (t < C) {
                        Shared* o = cluster.map_shared_rank(&sh, t);
                        o->cut = c;
                        o->draw = d;
                    }
                }
                cluster.sync();
                cut = sh.cut;
                found = cut.again == 0;
                drawn = found && set.min_p == 0.f;
                if (cut.again) {  // once more, by weight, among the larger values
                    by_count = false;
                    target = cut.target;
                    unit = (float)kWhole * kUnit / (float)cut.total;
                    lo = cut.above + 1;
                    hi = ordered(m);
                    above = 0;
                }
            } else if (lo == hi) {
                // one value: its first `j` ids are kept
                const uint64_t one = fixed(weight_of(unordered(hi)));
                uint64_t j = by_count ? target - above_count : (target - above + one - 1) / one;
                if (by_count && set.top_p < 1.f) {
                    const uint64_t z = above + j * one, goal = reached_at(set.top_p, z);
                    if (goal <= above) {
                        by_count = false;
                        target = goal;
                        unit = (float)kWhole * kUnit / (float)z;
                        lo = hi + 1;
                        hi = ordered(m);
                        above = 0;
                        continue;
                    }
                    if (one) j = min(j, (goal - above + one - 1) / one);
                }
                // the j-th of them, counted by warp in the order of the ids
                uint32_t here = 0;
                visit(unordered(hi), unordered(hi), [&](uint32_t e0, uint32_t e1, float, float) { here += (e0 != kAll) + (e1 != kAll); });
                here = __reduce_add_sync(0xFFFFFFFFu, here);
                cluster.sync();  // (the sums have been read)
                tell_warp(here);
                cluster.sync();
                uint64_t before_me = 0;
                for (uint32_t k = 0; k < rank * kWarps + warp; ++k) before_me += sh.warp_sum[k];
                if (before_me < j && j <= before_me + here) {
                    uint32_t left = (uint32_t)(j - before_me);
                    for (uint32_t v0 = 0; v0 < vecs && left; v0 += 32) {
                        const uint32_t v = v0 + lane;
                        uint32_t take = 0;
                        if (v < vecs) {
                            float f[VEC];
                            widen(mine[v], f, T());
#pragma unroll
                            for (uint32_t i = 0; i < VEC; ++i) take |= (ordered(f[i]) == hi ? 1u : 0u) << i;
                        }
                        const uint32_t c = __popc(take), cum = warp_scan(c), sum = __shfl_sync(0xFFFFFFFFu, cum, 31);
                        if (left > sum) {
                            left -= sum;
                            continue;
                        }
                        if (cum >= left && cum - c < left) {
                            for (uint32_t skip = left - (cum - c) - 1; skip; --skip) take &= take - 1;
                            const uint32_t id = id_of(v * VEC + __ffs(take) - 1);
                            for (uint32_t k = 0; k < C; ++k) cluster.map_shared_rank(&sh, k)->cut.id = id;
                        }
                        left = 0;
                    }
                }
                cluster.sync();
                cut = {hi, sh.cut.id, 0, 0, 0, 0};
                found = true;
            } else if (by_count || range.narrowed || !range.more) {
                // once more; what is left of the weights makes the whole
                unit *= range.grow;
            } else {
                // a few values of many tokens: on which side of the first bin's end? (the weights down to there tell)
                Weight s = {0.f, 0.f};
                visit(unordered(range.end), m, [&](uint32_t, uint32_t, float f0, float f1) {
                    add(s, weight_of(f0));
                    add(s, weight_of(f1));
                });
                cluster.sync();  // (the sums told before have been read)
                const uint64_t upto_end = cluster_total(fixed(s));
                if (upto_end >= target) {
                    lo = range.end;
                } else {
                    hi = range.end - 1;
                    above = upto_end;
                }
            }
        }
        if (least > cut.key) cut = {least, kAll, 0, 0, 0, 0};
    }

    // ---- 5. the kept weights by warp, in the order of the ids, and the draw
    const auto kept = [&](float f, uint32_t id) {
        const uint32_t key = ordered(f);
        return !(key < cut.key || (key == cut.key && id > cut.id));
    };
    if (!drawn) {
        Weight s = {0.f, 0.f};
        if (cut.key == kLowest && set.min_p == 0.f) {
            add_all(s);
        } else {
            visit(unordered(cut.key), m, [&](uint32_t e0, uint32_t e1, float f0, float f1) {
                const Weight a = weight_of(e0 != kAll && kept(f0, id_of(e0)) ? f0 : -kInf);
                const Weight b = weight_of(e1 != kAll && kept(f1, id_of(e1)) ? f1 : -kInf);
                if (enough(a)) add(s, a);
                if (enough(b)) add(s, b);
            });
        }
        const uint64_t sum = warp_total(fixed(s));
        tell_warp(sum);
        cluster.sync();
    }
    // (no one writes to or reads from other CTAs from here on)
    const Draw draw = drawn ? sh.draw : draw_warp();
    if (draw.warp / kWarps != rank) return;
    // The CTA that has it walks the warp's part, a few neighbours to a thread.
    bool exact;
    const uint64_t want = part_of(set.u, draw.z, &exact) - draw.start;
    const uint32_t each = (vecs + kThreads - 1) / kThreads, from = (draw.warp % kWarps) * vecs, number = draw.warp * p.chunk - before;
    const uint32_t v_begin = min(t * each, vecs), v_end = min(v_begin + each, vecs);
    const auto weights = [&](uint32_t v, uint64_t (&w)[VEC], float (&f)[VEC]) {
        widen(slice[from + v], f, T());
#pragma unroll
        for (uint32_t i = 0; i < VEC; ++i) {
            const Weight q = weight_of(kept(f[i], number + v * VEC + i) ? f[i] : -kInf);
            w[i] = enough(q) ? fixed(q) : 0;
        }
    };
    uint64_t here = 0, all;
    for (uint32_t v = v_begin; v < v_end; ++v) {
        float f[VEC];
        uint64_t w[VEC];
        weights(v, w, f);
#pragma unroll
        for (uint32_t i = 0; i < VEC; ++i) here += w[i];
    }
    const uint64_t below = block_scan(here, sh.scan, &all) - here;
    // (these sums are rounded another way than the warp's: at its very end the last kept is meant)
    uint64_t left = min(want, all - 1);
    if (left < below || left >= below + here) return;
    left -= below;
    for (uint32_t v = v_begin; v < v_end; ++v) {
        float f[VEC];
        uint64_t w[VEC];
        weights(v, w, f);
#pragma unroll
        for (uint32_t i = 0; i < VEC; ++i) {
            if (left < w[i]) {
                token_is(number + v * VEC + i, f[i], draw.z);
                return;
            }
            left -= w[i];
        }
    }
}

constexpr uint32_t vecs_of(uint32_t V, uint32_t ctas, uint32_t vec) {  // of a warp
    return (V + vec - 1 + ctas * kWarps * vec - 1) / (ctas * kWarps * vec);
}
static_assert(vecs_of(LP_MAX_SAMPLE_VOCAB, kMaxCluster, 4) * kWarps * 16 + sizeof(Shared) <= 227 * 1024, "the longest rows fit");

template <typename T>
lp_status launch_sample(SampleParams p, lp_stream_t stream) {
    constexpr uint32_t kVec = Vec<T>::kElems;
    static std::atomic<uint64_t> smem_set;
    // CTAs of a row: slices of about 16384 elements at most (the smallest number that gives them), eight at most
    uint32_t c = 1;
    while (c < kMaxCluster && p.V > c * 16384) c *= 2;
    const uint32_t vecs = vecs_of(p.V, c, kVec);
    p.chunk = vecs * kVec;
    auto kernel = k_sample<T>;
    constexpr size_t kMost = (size_t)vecs_of(LP_MAX_SAMPLE_VOCAB, kMaxCluster, kVec) * kWarps * 16;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), kMost, &smem_set)) return LP_ERR_CUDA;
    return launch(kernel, dim3(p.T * c), kThreads, (size_t)vecs * kWarps * 16, stream, c, p);
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
