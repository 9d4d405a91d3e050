// Draw of the next token (include/lp_head.h): temperature, top-k, top-p and min-p, from a given
// random number a row.
//
// A row belongs to a cluster of up to eight CTAs, each with a slice of it in shared memory, read
// from HBM once. Weights exp((x - max) / tau) are formed with about 40 correct bits (a table of 64
// powers and a short series, in pairs of f32, two tokens to an instruction) and added as pairs or as
// integers of 2^-43: the token is a comparison of sums of up to some hundred thousand weights with
// each other, and f32's rounding would move it in a few rows of a hundred. All three filters keep a
// prefix of the order (value descending, id ascending), so that what is kept is told by the last
// kept (value, id):
//   top-k: each CTA tells a value that enough of its threads' largest reach (a coarse histogram);
//          what lies above the least of these is listed and ranked by the cluster's first CTA.
//   top-p: what weighs less than (1 - p) Z / V is never kept. Where Z is small the rest is listed
//          as well; else, or if it does not fit, a histogram over the values' bits finds the bin
//          in which p Z is reached, and that bin is listed. A bin of more than fits is cut again;
//          one that holds a single value is cut by id.
// The draw follows the ids: the kept weights are summed by warp, and the CTA in which u Z falls
// walks that warp's part once more. CTAs write what the others need into their shared memory
// before a barrier of the cluster.
#include <cooperative_groups.h>

#include "lp_head_common.h"

namespace {

using namespace lph;
namespace cg = cooperative_groups;

constexpr uint32_t kThreads = 384, kWarps = kThreads / 32;
constexpr uint32_t kResident = 3;  // CTAs per SM, with slices of up to 16384 f32
constexpr uint32_t kMaxCluster = 8;
constexpr uint32_t kList = 512;    // tokens that are ranked
constexpr uint32_t kBins = kThreads;
constexpr uint32_t kBound = 256;
constexpr uint32_t kTable = 64;
constexpr uint32_t kLowest = 0x00800000u;  // ordered() of the lowest finite value
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kPoint = 43;           // weights as integers: 2^43 is that of the largest
constexpr float kUnit = 8796093022208.f, kInvUnit = 1.1368683772161603e-13f;  // 2^43, 2^-43
constexpr float kSmallest = 40.f;    // -log2 of the smallest weight that counts
constexpr float kFewWeights = 8.f;   // Z up to which a top-p row's tokens are listed at once
constexpr uint32_t kCount = 384;     // tokens up to which ranks are counted, and not sorted

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
    uint32_t again;        // the search goes on among keys above `above`, for the weight `target`
    uint32_t above;
    uint64_t target;
};

struct Told {              // by each CTA
    float top;             // its largest value
    uint32_t share, whole; // keys that ceil(k / CTAs), and k, of its threads' largest reach
};

struct Shared {
    union {
        uint64_t list[kList];    // key << 32 | ~id
        uint32_t bound[kBound];  // (before the list)
    };
    union {
        struct {
            uint32_t count[kBins], low[kBins], high[kBins];
        };
        uint64_t stage[kList + kList / 2];  // a CTA's part of the list; the ranked list, and its keys
    };
    float2 table[kTable];
    uint64_t scan[kWarps];
    uint64_t warp_sum[kMaxCluster * kWarps];
    uint64_t cta_sum[kMaxCluster];
    uint64_t words[4];
    Told told[kMaxCluster];
    Setting set;
    Cut cut;
    uint32_t listed, staged, place;
    uint32_t found_bin, found_count, found_before_count;
    uint64_t found_before, found_weight;
};

// 2^(j / 64) as pairs of f32, at compile time: by repeated products of 2^(1 / 64), whose digits a
// series of the exponential gives.
struct Table {
    float hi[kTable], lo[kTable];
};
constexpr Table make_table() {
    Table t = {};
    for (uint32_t j = 0; j < kTable; ++j) {
        const double y = 0.6931471805599453094 * j / kTable;
        double term = 1.0, sum = 0.0;
        for (int n = 30; n > 0; --n) {  // smallest terms first
            term = 1.0;
            for (int k = 1; k <= n; ++k) term *= y / k;
            sum += term;
        }
        sum += 1.0;
        t.hi[j] = (float)sum;
        t.lo[j] = (float)(sum - (double)(float)sum);
    }
    return t;
}
__constant__ Table c_table = make_table();

// Two f32 at a time.
using f2 = uint64_t;
__device__ __forceinline__ f2 both(float a, float b) { return (f2)__float_as_uint(a) | (f2)__float_as_uint(b) << 32; }
__device__ __forceinline__ f2 both(float a) { return both(a, a); }
__device__ __forceinline__ float first(f2 a) { return __uint_as_float((uint32_t)a); }
__device__ __forceinline__ float second(f2 a) { return __uint_as_float((uint32_t)(a >> 32)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 sub2(f2 a, f2 b) { return fma2(b, both(-1.f), a); }

struct Scale {             // of a row
    float m, low;          // largest value; values below `low` weigh 0
    f2 neg_m, chi, neg_chi, clo;
};
__device__ __forceinline__ Scale scale_of(float m, const Setting& s) {
    // where exp is below 2^-40 (or f32 ends): low - m and its products stay finite
    const float low = fmaxf(fmaxf(m - 28.5f * s.tau, m - 3e38f), -3.402823466e38f);
    return {m, low, both(-m), both(s.chi), both(-s.chi), both(s.clo)};
}

struct Weight2 {
    f2 hi, lo;  // hi + lo; hi is rounded to 24 bits
};
// exp((x - m) / tau) of two values; 0 below 2^-40.
__device__ __forceinline__ Weight2 weigh(float x0, float x1, const Scale& r, const float2* table) {
    const f2 x = both(fmaxf(x0, r.low), fmaxf(x1, r.low));
    const f2 d = add2(x, r.neg_m), back = sub2(d, x);
    const f2 err = add2(sub2(x, sub2(d, back)), sub2(r.neg_m, back));  // x - m = d + err
    const f2 np = mul2(d, r.neg_chi);
    const f2 rest = fma2(err, r.chi, fma2(d, r.clo, fma2(d, r.chi, np)));
    // -np + rest = log2 of the weight = k / 64 + g; an ulp of 1.5 * 2^17 is 1 / 64
    const f2 magic = both(196608.f);
    const f2 t = sub2(magic, np);
    const f2 g = sub2(rest, add2(np, sub2(t, magic)));
    // 2^g - 1 = g ln 2 + (g ln 2)^2 / 2 + ...; the first term as a pair
    const f2 l1 = both(0.693147180559945f);
    const f2 qh = mul2(g, l1);
    f2 ql = fma2(g, l1, mul2(g, both(-0.693147180559945f)));
    ql = fma2(g, both(-1.9046542e-9f), ql);
    const f2 series = fma2(g, fma2(g, both(0.00961812910762848f), both(0.0555041086648216f)), both(0.240226506959101f));
    ql = fma2(mul2(g, g), series, ql);
    const uint32_t k0 = (uint32_t)t, k1 = (uint32_t)(t >> 32);
    const float2 t0 = table[k0 & (kTable - 1)], t1 = table[k1 & (kTable - 1)];
    const f2 th = both(t0.x, t1.x), tl = both(t0.y, t1.y);
    const f2 a = mul2(th, qh), b = fma2(th, qh, mul2(th, mul2(qh, both(-1.f))));
    const f2 s = add2(th, a);
    const f2 e = add2(add2(sub2(th, s), a), fma2(th, ql, fma2(tl, qh, add2(tl, b))));
    // 2^(k >> 6): the bits of t are 0x48400000 + k
    const auto power = [&r](uint32_t bits, float neg, float x) {
        const uint32_t p = ((bits << 17) & 0xFF800000u) + ((127u - 0x1210000u) << 23);
        return neg <= kSmallest && x >= r.low ? __uint_as_float(p) : 0.f;
    };
    const f2 scale = both(power(k0, first(np), x0), power(k1, second(np), x1));
    return {mul2(s, scale), mul2(e, scale)};
}
__device__ __forceinline__ uint64_t fixed(float hi, float lo) {
    return __float2ull_rn(hi * kUnit) + (uint64_t)__float2ll_rn(lo * kUnit);
}
__device__ __forceinline__ uint64_t fixed(Weight2 w) { return fixed(first(w.hi), first(w.lo)) + fixed(second(w.hi), second(w.lo)); }
// Sums of weights, as pairs.
__device__ __forceinline__ void add(Weight2& s, Weight2 w) {
    const f2 t = add2(s.hi, w.hi), z = sub2(t, s.hi);
    s.lo = add2(s.lo, add2(add2(sub2(s.hi, sub2(t, z)), sub2(w.hi, z)), w.lo));
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

// n keys (n <= kList) of `from` in descending order, to `to`. Few are ranked by counting the
// larger ones (one to eight threads a key), many by a bitonic sort (384: 3.3 against 3.6 us).
__device__ __forceinline__ void sort_list(uint64_t* from, uint64_t* to, uint32_t n) {
    const uint32_t t = threadIdx.x;
    if (n <= kCount) {
        const uint32_t shift = n <= kCount / 8 ? 3 : n <= kCount / 4 ? 2 : n <= kCount / 2 ? 1 : 0;
        const uint32_t at = t >> shift, parts = 1u << shift;
        const uint64_t key = at < n ? from[at] : 0;
        uint32_t rank = 0;
#pragma unroll 4
        for (uint32_t j = t & (parts - 1); j < n; j += parts) rank += from[j] > key;
        for (uint32_t k = 1; k < parts; k *= 2) rank += __shfl_xor_sync(0xFFFFFFFFu, rank, k);
        if (at < n && (t & (parts - 1)) == 0) to[rank] = key;
        __syncthreads();
        return;
    }
    for (uint32_t i = t; i < kList; i += kThreads) to[i] = i < n ? from[i] : 0;
    __syncthreads();
    for (uint32_t k = 2; k <= kList; k *= 2)
        for (uint32_t j = k / 2; j > 0; j /= 2) {
            if (t < kList / 2) {
                const uint32_t i = 2 * j * (t / j) + t % j;
                const uint64_t a = to[i], b = to[i + j];
                if ((a < b) == ((i & k) == 0)) {
                    to[i] = b;
                    to[i + j] = a;
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

__device__ __forceinline__ Setting setting_of(const SampleParams& p, uint32_t row, bool report) {
    Setting s = {};
    const int b = request_of(p.row_offsets, p.B, row);
    if (b < 0) {
        if (report) flag(p.status, LP_ERR_OFFSETS);
        return s;
    }
    float tau = p.temperature ? p.temperature[b] : 1.f;
    const float top_p = p.top_p ? p.top_p[b] : 1.f, min_p = p.min_p ? p.min_p[b] : 0.f, u = p.uniform[row];
    const int k = p.top_k ? p.top_k[b] : 0;
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
    if (t < kTable) sh.table[t] = make_float2(c_table.hi[t], c_table.lo[t]);
    if (t < kBound) sh.bound[t] = 0;
    if (t == 0) sh.staged = sh.listed = 0;
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // (waited for before others' memory is written to)
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

    // ---- 1. read; the setting, by the last warp; the largest value, threads' largest in coarse bins
    if (t == kThreads - 1) sh.set = setting_of(p, row, rank == 0);
    __syncwarp();
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
        for (uint32_t i = 0; i < VEC; ++i) top = max_nan(top, f[i]);
    }
    __syncthreads();  // the bins are cleared, the setting is there
    const Setting set = sh.set;
    if (set.k && top > -kInf) atomicAdd(&sh.bound[bound_bin(top)], 1);
#pragma unroll
    for (int k = 16; k > 0; k /= 2) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
    if (lane == 0) reinterpret_cast<float*>(sh.scan)[warp] = top;
    __syncthreads();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (warp == 0) {
        Told told;
        top = lane < kWarps ? reinterpret_cast<float*>(sh.scan)[lane] : -kInf;
#pragma unroll
        for (int k = 8; k > 0; k /= 2) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, k));
        told.top = __shfl_sync(0xFFFFFFFFu, top, 0);
        told.share = told.whole = kLowest;
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
    float m = -kInf;
    uint32_t lo = kAll, lo_whole = kLowest;  // keys below `lo` are not kept
    for (uint32_t k = 0; k < C; ++k) {
        m = max_nan(m, sh.told[k].top);
        lo = min(lo, sh.told[k].share);
        lo_whole = max(lo_whole, sh.told[k].whole);
    }
    lo = max(lo, lo_whole);
    if (!set.ok || !(m > -kInf && m < kInf)) {
        if (rank == 0 && t == 0) {
            if (set.ok) flag(p.status, LP_ERR_LOGITS);
            p.out[row] = kAll;
            if (p.out_logprob) p.out_logprob[row] = __uint_as_float(0x7FC00000u);
        }
        return;
    }
    const Scale scale = scale_of(m, set);
    uint32_t hi = ordered(m);
    // min-p: what weighs less than that is not kept. `least` is a key below all that are (room for
    // the roundings here), the weights decide.
    uint32_t least = kLowest;
    if (set.min_p > 0.f) {
        const float f = m + set.tau * (__logf(set.min_p) - 0.01f) - fabsf(m) * 1e-6f;
        least = f > -3e38f ? min(max(ordered(f + 0.f), kLowest), hi) : kLowest;
    }
    const auto enough = [&](float w_hi, float w_lo) {  // (hi is the pair rounded to f32)
        return w_hi > set.min_p || (w_hi == set.min_p && w_lo >= 0.f);
    };
    const auto token_is = [&](uint32_t id, float value, uint64_t z) {
        p.out[row] = id;
        if (p.out_logprob) {
            // the largest value is kept: z >= 2^43, and both terms have one sign
            const float lnz = log1pf((float)(z - (1ull << kPoint)) * kInvUnit);
            p.out_logprob[row] = (value - m) / set.tau - lnz;
        }
    };
    // Weights of places 2 t and 2 t + 1 of the ranked list (0 from `n` on), and whether min-p keeps them.
    const auto list_weights = [&](uint32_t n, uint64_t (&w)[2], bool (&fine)[2]) {
        const float f0 = 2 * t < n ? unordered((uint32_t)(sh.stage[2 * t] >> 32)) : -kInf;
        const float f1 = 2 * t + 1 < n ? unordered((uint32_t)(sh.stage[2 * t + 1] >> 32)) : -kInf;
        const Weight2 q = weigh(f0, f1, scale, sh.table);
        w[0] = fixed(first(q.hi), first(q.lo));
        w[1] = fixed(second(q.hi), second(q.lo));
        fine[0] = w[0] && enough(first(q.hi), first(q.lo));
        fine[1] = w[1] && enough(second(q.hi), second(q.lo));
    };
    // All weights of the warp's elements.
    const auto add_all = [&](Weight2& s) {
#pragma unroll 1
        for (uint32_t v = lane; v < vecs; v += 32) {
            float f[VEC];
            widen(mine[v], f, T());
            float high = f[0];
#pragma unroll
            for (uint32_t i = 1; i < VEC; ++i) high = fmaxf(high, f[i]);
            if (!__any_sync(__activemask(), high >= scale.low)) continue;
#pragma unroll
            for (uint32_t i = 0; i < VEC; i += 2) add(s, weigh(f[i], f[i + 1], scale, sh.table));
        }
    };
    // Visits the warp's elements whose keys lie in [from, to], two at a time: body(element, element or
    // kAll, value, value). Lanes take them out of masks of 32, so that few cost little.
    const auto visit = [&](uint32_t from, uint32_t to, auto body) {
        for (uint32_t v0 = 0; v0 < vecs; v0 += 32 * (32 / VEC)) {
            uint32_t take = 0;
#pragma unroll
            for (uint32_t j = 0; j < 32 / VEC; ++j) {
                const uint32_t v = v0 + j * 32 + lane;
                if (v < vecs) {
                    float f[VEC];
                    widen(mine[v], f, T());
#pragma unroll
                    for (uint32_t i = 0; i < VEC; ++i) {
                        const uint32_t key = ordered(f[i]);
                        take |= (key >= from && key <= to ? 1u : 0u) << (j * VEC + i);
                    }
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

    Shared* lead = cluster.map_shared_rank(&sh, 0);
    // Tokens with keys in [from, to] into the first CTA's list; true where all of them fit. Ends with a
    // barrier of the cluster.
    const auto make_list = [&](uint32_t from, uint32_t to) {
        visit(from, to, [&](uint32_t e0, uint32_t e1, float f0, float f1) {
            const uint32_t n = (e0 != kAll) + (e1 != kAll), upto = warp_scan(n);
            uint32_t at = 0;
            if (lane == 31) at = atomicAdd(&sh.staged, upto);
            at = __shfl_sync(0xFFFFFFFFu, at, 31) + upto - n;
            if (e0 != kAll && at < kList) sh.stage[at] = (uint64_t)ordered(f0) << 32 | (uint32_t)~id_of(e0);
            if (e1 != kAll && at + 1 < kList) sh.stage[at + 1] = (uint64_t)ordered(f1) << 32 | (uint32_t)~id_of(e1);
        });
        __syncthreads();
        const uint32_t n = sh.staged;
        if (t == 0) sh.place = n ? atomicAdd(&lead->listed, n) : 0u;
        __syncthreads();
        const uint32_t place = sh.place;
        if (place <= kList && n <= kList - place)
            for (uint32_t i = t; i < n; i += kThreads) lead->list[place + i] = sh.stage[i];
        cluster.sync();
    };

    Cut cut = {least, kAll, 0, 0, 0};
    if (set.k || set.top_p < 1.f) {
        uint64_t target = set.k;
        bool by_count = set.k != 0, few = set.k <= kList;
        if (!by_count) {
            // ---- 2. the sum of all weights, and from it a bound
            Weight2 s = {0, 0};
            add_all(s);
            uint64_t all;
            (void)block_scan(fixed(s), sh.scan, &all);
            if (t < C) cluster.map_shared_rank(&sh, t)->cta_sum[rank] = all;
            cluster.sync();
            uint64_t z = 0;
            for (uint32_t k = 0; k < C; ++k) z += sh.cta_sum[k];
            target = reached_at(set.top_p, z);
            const float sum = (float)z * kInvUnit;
            // kept tokens weigh (1 - p) Z / V at least (with room for the roundings here)
            const float f = m + set.tau * (__logf((1.f - set.top_p) * sum / (float)p.V) - 0.01f) - fabsf(m) * 1e-6f;
            lo = f > -3e38f ? min(max(ordered(f + 0.f), kLowest), hi) : kLowest;
            few = sum < kFewWeights;
        }
        // ---- 3. all that can be kept in one list?
        if (few) {
            make_list(lo, hi);
            const uint32_t n = lead->listed;
            if (n <= kList) {
                // the first CTA does the rest; the others have read its count, and no one reads theirs
                if (rank != 0) {
                    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
                    return;
                }
                sort_list(sh.list, sh.stage, n);
                uint64_t w[2], all;
                bool fine[2];
                const uint32_t at0 = 2 * t;
                list_weights(set.k ? min(n, set.k) : n, w, fine);
                uint64_t below = block_scan(w[0] + w[1], sh.scan, &all) - (w[0] + w[1]);
                if (by_count) target = set.top_p < 1.f ? reached_at(set.top_p, all) : ~0ull;
                uint32_t keep = 0;
#pragma unroll
                for (uint32_t i = 0; i < 2; ++i) {
                    keep += fine[i] && below < target;
                    below += w[i];
                    if (at0 + i < n) sh.list[at0 + i] = w[i];  // (the list is in `stage` now)
                }
                uint64_t kept;
                (void)block_scan(keep, sh.scan, &kept);
                // The first `kept` of them, in the order of their ids: what lies below each.
                uint64_t z = 0;
                bool exact;
                if (kept <= kCount) {
                    const uint32_t n_kept = (uint32_t)kept;
                    const uint32_t shift = n_kept <= kCount / 8 ? 3 : n_kept <= kCount / 4 ? 2 : n_kept <= kCount / 2 ? 1 : 0;
                    const uint32_t at = t >> shift, parts = 1u << shift;
                    const uint64_t entry = at < n_kept ? sh.stage[at] : 0;
                    const uint32_t not_id = (uint32_t)entry;
                    uint64_t under = 0;
#pragma unroll 4
                    for (uint32_t j = t & (parts - 1); j < n_kept; j += parts) {
                        const uint64_t wj = sh.list[j];
                        under += (uint32_t)sh.stage[j] > not_id ? wj : 0;
                        z += wj;
                    }
                    for (uint32_t k = 1; k < parts; k *= 2) {
                        under += __shfl_xor_sync(0xFFFFFFFFu, under, k);
                        z += __shfl_xor_sync(0xFFFFFFFFu, z, k);
                    }
                    const uint64_t want = part_of(set.u, z, &exact);
                    if (at < n_kept && (t & (parts - 1)) == 0 && under <= want && want < under + sh.list[at])
                        token_is(~not_id, unordered((uint32_t)(entry >> 32)), z);
                } else {
                    // sorted by id, with their places; keys and weights are looked up there
                    uint32_t* keys = reinterpret_cast<uint32_t*>(sh.stage + kList);
                    uint64_t order[2];
#pragma unroll
                    for (uint32_t i = 0; i < 2; ++i) {
                        const uint32_t at = at0 + i;
                        order[i] = at < kept ? sh.stage[at] << 32 | at : 0;
                        if (at < kList) keys[at] = (uint32_t)(sh.stage[at] >> 32);
                    }
                    uint64_t mine2[2] = {at0 < kept ? sh.list[at0] : 0, at0 + 1 < kept ? sh.list[at0 + 1] : 0};
                    __syncthreads();
#pragma unroll
                    for (uint32_t i = 0; i < 2; ++i)
                        if (at0 + i < kList) sh.list[at0 + i] = order[i];
                    __syncthreads();
                    sort_list(sh.list, sh.stage, (uint32_t)kept);
                    // (weights back where their places are)
#pragma unroll
                    for (uint32_t i = 0; i < 2; ++i)
                        if (at0 + i < kList) sh.list[at0 + i] = mine2[i];
                    __syncthreads();
                    uint64_t own = 0;
                    uint32_t place[2];
#pragma unroll
                    for (uint32_t i = 0; i < 2; ++i) {
                        place[i] = at0 + i < kept ? (uint32_t)sh.stage[at0 + i] : 0u;
                        w[i] = at0 + i < kept ? sh.list[place[i]] : 0;
                        own += w[i];
                    }
                    uint64_t under = block_scan(own, sh.scan, &z) - own;
                    const uint64_t want = part_of(set.u, z, &exact);
#pragma unroll
                    for (uint32_t i = 0; i < 2; ++i) {
                        if (w[i] && under <= want && want < under + w[i])
                            token_is(~(uint32_t)(sh.stage[at0 + i] >> 32), unordered(keys[place[i]]), z);
                        under += w[i];
                    }
                }
                asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
                return;
            }
        }
        // ---- 4. the value at which the target is reached, by histograms over [lo, hi]
        bool cut_found = false, read = few;  // whether others may still read the tables and the list
        for (int round = 0; round < 2 && !cut_found; ++round) {
            uint64_t above = 0;           // weight of the keys above hi
            uint32_t above_count = 0;
            for (;;) {
                uint32_t shift = 0;
                while ((hi - lo) >> shift >= kBins) ++shift;
                if (read) cluster.sync();
                read = true;
                sh.count[t] = sh.low[t] = sh.high[t] = 0;
                if (t == 0) {
                    sh.listed = sh.staged = 0;
                    sh.found_bin = kAll;
                }
                __syncthreads();
                visit(lo, hi, [&](uint32_t e0, uint32_t e1, float f0, float f1) {
                    const Weight2 w = weigh(f0, f1, scale, sh.table);
                    const auto count = [&](float f, uint64_t fix) {
                        const uint32_t bin = (hi - ordered(f)) >> shift;
                        atomicAdd(&sh.count[bin], 1);
                        const uint32_t was = atomicAdd(&sh.low[bin], (uint32_t)fix);
                        const uint32_t up = (uint32_t)(fix >> 32) + (was + (uint32_t)fix < was);
                        if (up) atomicAdd(&sh.high[bin], up);
                    };
                    if (e0 != kAll) count(f0, fixed(first(w.hi), first(w.lo)));
                    if (e1 != kAll) count(f1, fixed(second(w.hi), second(w.lo)));
                });
                cluster.sync();
                uint32_t n = 0;
                uint64_t w = 0, all_w, all_n;
                for (uint32_t k = 0; k < C; ++k) {
                    const Shared* o = cluster.map_shared_rank(&sh, k);
                    n += o->count[t];
                    w += (uint64_t)o->high[t] << 32 | o->low[t];
                }
                const uint64_t upto = block_scan(w, sh.scan, &all_w), upto_n = block_scan(n, sh.scan, &all_n);
                const uint64_t have = by_count ? above_count + upto_n : above + upto, step = by_count ? n : w;
                if (have >= target && have - step < target) {
                    sh.found_bin = t;
                    sh.found_count = n;
                    sh.found_before = above + upto - w;
                    sh.found_before_count = above_count + (uint32_t)(upto_n - n);
                    sh.found_weight = w;
                }
                __syncthreads();
                const uint32_t bin = sh.found_bin;
                if (bin == kAll) {  // all of it is kept (k is more than there are)
                    if (by_count && set.top_p < 1.f) {
                        cut.above = lo - 1;
                        cut.target = reached_at(set.top_p, above + all_w);
                    } else {
                        cut = {max(lo, least), kAll, 0, 0, 0};
                        cut_found = true;
                    }
                    break;
                }
                above = sh.found_before;
                above_count = sh.found_before_count;
                const uint32_t in_bin = sh.found_count;
                const uint64_t bin_weight = sh.found_weight;
                hi = hi - (bin << shift);
                lo = max(lo, hi - (1u << shift) + 1 > hi ? 0u : hi - (1u << shift) + 1);
                if (in_bin > kList && lo < hi) continue;
                if (in_bin > kList) {
                    // one value: its first `j` ids are kept
                    const uint64_t each = bin_weight / in_bin;
                    uint64_t j = by_count ? target - above_count : (target - above + each - 1) / each;
                    if (by_count && set.top_p < 1.f) {
                        const uint64_t next = reached_at(set.top_p, above + j * each);
                        if (next <= above) {
                            cut.above = hi;
                            cut.target = next;
                            break;
                        }
                        if (each) j = min(j, (next - above + each - 1) / each);
                    }
                    // the j-th of them, counted by warp in the order of the ids
                    uint32_t here = 0;
                    visit(hi, hi, [&](uint32_t e0, uint32_t e1, float, float) { here += (e0 != kAll) + (e1 != kAll); });
                    here = __reduce_add_sync(0xFFFFFFFFu, here);
                    if (lane < C) cluster.map_shared_rank(&sh, lane)->warp_sum[rank * kWarps + warp] = here;
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
                            const uint32_t c = __popc(take), cum = warp_scan(c), all = __shfl_sync(0xFFFFFFFFu, cum, 31);
                            if (left > all) {
                                left -= all;
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
                    cut = {hi, sh.cut.id, 0, 0, 0};
                } else {
                    // the bin's tokens, ranked by the first CTA (its tables have been read before it stages)
                    cluster.sync();
                    make_list(lo, hi);
                    if (rank == 0) {
                        sort_list(sh.list, sh.stage, in_bin);
                        const uint32_t limit = by_count ? (uint32_t)(target - above_count) : kAll, at0 = 2 * t;
                        uint64_t w2[2], all;
                        bool fine[2];
                        list_weights(min(in_bin, limit), w2, fine);
                        uint64_t below = above + block_scan(w2[0] + w2[1], sh.scan, &all) - (w2[0] + w2[1]);
                        uint64_t reach = target;
                        if (by_count) reach = set.top_p < 1.f ? reached_at(set.top_p, above + all) : ~0ull;
                        uint32_t keep = 0;
#pragma unroll
                        for (uint32_t i = 0; i < 2; ++i) {
                            keep += at0 + i < in_bin && at0 + i < limit && below < reach;
                            below += w2[i];
                        }
                        uint64_t kept;
                        (void)block_scan(keep, sh.scan, &kept);
                        if (t < C) {
                            Cut c = {kAll, 0, 1, hi, reach};  // reached among larger values
                            if (kept) {
                                const uint64_t last = sh.stage[kept - 1];
                                c = {(uint32_t)(last >> 32), ~(uint32_t)last, 0, 0, 0};
                            }
                            cluster.map_shared_rank(&sh, t)->cut = c;
                        }
                    }
                    cluster.sync();
                    cut = sh.cut;
                    if (cut.again) break;
                }
                cut_found = true;
                if (least > cut.key) cut = {least, kAll, 0, 0, 0};
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
    const auto kept_weight = [&](uint32_t key, uint32_t id, float w_hi, float w_lo) {
        return key < cut.key || (key == cut.key && id > cut.id) || !enough(w_hi, w_lo) ? 0ull : fixed(w_hi, w_lo);
    };
    uint64_t sum;
    {
        Weight2 s = {0, 0};
        if (cut.key == kLowest && set.min_p == 0.f) {  // all
            add_all(s);
        } else {
            visit(cut.key, kAll, [&](uint32_t e0, uint32_t e1, float f0, float f1) {
                if (e0 != kAll && ordered(f0) == cut.key && id_of(e0) > cut.id) f0 = -kInf;
                if (e1 != kAll && ordered(f1) == cut.key && id_of(e1) > cut.id) f1 = -kInf;
                Weight2 w = weigh(f0, f1, scale, sh.table);
                if (set.min_p > 0.f) {
                    const f2 keep = both(enough(first(w.hi), first(w.lo)) ? 1.f : 0.f, enough(second(w.hi), second(w.lo)) ? 1.f : 0.f);
                    w = {mul2(w.hi, keep), mul2(w.lo, keep)};
                }
                add(s, w);
            });
        }
        sum = fixed(s);
#pragma unroll
        for (int k = 16; k > 0; k /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
    }
    if (lane < C) cluster.map_shared_rank(&sh, lane)->warp_sum[rank * kWarps + warp] = sum;
    cluster.sync();
    // (no one writes to or reads from other CTAs from here on)
    constexpr uint32_t kEach = kMaxCluster * kWarps / 32;  // of the warps' sums to a lane
    uint64_t part[kEach], own = 0;
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
        const uint32_t g = lane * kEach + i;
        part[i] = g < C * kWarps ? sh.warp_sum[g] : 0;
        own += part[i];
    }
    const uint64_t upto = warp_scan(own), z = __shfl_sync(0xFFFFFFFFu, upto, 31);
    bool exact;
    const uint64_t want = part_of(set.u, z, &exact);
    uint64_t below = upto - own, start = 0;
    uint32_t hit = kAll;
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
        if (below <= want && want < below + part[i]) {
            hit = lane * kEach + i;
            start = below;
        }
        below += part[i];
    }
    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, hit != kAll)) - 1;  // (one lane: want < z)
    hit = __shfl_sync(0xFFFFFFFFu, hit, src);
    start = __shfl_sync(0xFFFFFFFFu, start, src);
    if (hit / kWarps != rank) return;
    // The CTA that has it walks the warp's part, a few neighbours to a thread.
    const uint32_t each = (vecs + kThreads - 1) / kThreads, from = (hit % kWarps) * vecs, number = hit * p.chunk - before;
    const uint32_t v_begin = min(t * each, vecs), v_end = min(v_begin + each, vecs);
    const auto weights = [&](uint32_t v, uint64_t (&w)[VEC], float (&f)[VEC]) {
        widen(slice[from + v], f, T());
#pragma unroll
        for (uint32_t i = 0; i < VEC; i += 2) {
            const Weight2 q = weigh(f[i], f[i + 1], scale, sh.table);
            const uint32_t id = number + v * VEC + i;
            w[i] = kept_weight(ordered(f[i]), id, first(q.hi), first(q.lo));
            w[i + 1] = kept_weight(ordered(f[i + 1]), id + 1, second(q.hi), second(q.lo));
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
    below = block_scan(here, sh.scan, &all) - here;
    // (these sums are rounded another way than the warp's: at its very end the last kept is meant)
    uint64_t left = min(want - start, all - 1);
    if (left < below || left >= below + here) return;
    left -= below;
    for (uint32_t v = v_begin; v < v_end; ++v) {
        float f[VEC];
        uint64_t w[VEC];
        weights(v, w, f);
#pragma unroll
        for (uint32_t i = 0; i < VEC; ++i) {
            if (left < w[i]) {
                token_is(number + v * VEC + i, f[i], z);
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
