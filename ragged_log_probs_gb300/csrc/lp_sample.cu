// Draw of the next token (include/lp_head.h): temperature, top-k, top-p and min-p, from a given
// random number a row.
//
// Two kernels. The first reads the logits once, at HBM's rate: a warp takes a part of 1024 tokens
// and writes down its largest value, and what the row's setting asks for: the sum of its weights
// (top-p, or no filter) or some of its lanes' largest values in order (top-k). The second kernel, a
// cluster of up to eight CTAs a row, decides from that what can be kept, and reads again only the
// parts that hold some of it, from L2 for the most part; without a filter that is the one part
// in which the token lies.
//
// Weights exp((x - max) / tau) are formed with about 34 correct bits (a table of 256 powers, and a
// short series for what is left of the exponent) and added as pairs of f32 or as integers of 2^-43:
// the token is a comparison of sums of up to some hundred thousand weights with each other, and
// f32's rounding would move it in a few rows of a hundred. All three filters keep a prefix of the
// order (value descending, id ascending), so that what is kept is told by the last kept (value, id):
//   top-k: a value that k tokens reach for sure is read from the parts' ordered values; what
//          lies above it is listed and ranked by the cluster's first CTA (k up to 384; above
//          that a histogram of counts lowers the number of those that pass first).
//   top-p: what weighs less than (1 - p) Z / V is never kept. Where that leaves few tokens they are
//          listed as well. Else, or if it does not fit, a histogram of f32 weights (31 bins over the
//          values) finds the bins in which p Z can be reached; what lies above them is summed
//          exactly, what lies in them is listed. Bins of more than fits are cut again; a single
//          value is cut by id.
// The draw follows the ids: the kept weights are summed by part, and the first CTA walks the part
// in which u Z falls. CTAs write what the others need into their shared memory before a barrier
// of the cluster.
//
// Measured: 256 rows of 128256 f32: best token 33 us, temperature 59, min-p 58, top-k with top-p 75,
// top-p alone 165, of every kind 92; the bytes once take 19. The first kernel is bound by HBM without
// weights (26 us), by its instructions with them (45, 78 % of the issue slots). The second is bound
// by latency: barriers of the cluster (some 1 us each) and what one CTA does for the others between
// them, 29 % of the issue slots, 14 % of HBM. One row: 12 to 30 us, of which 9 are the two launches
// and their reads.
#include <cooperative_groups.h>

#include <type_traits>

#include "lp_head_common.h"

namespace {

using namespace lph;
namespace cg = cooperative_groups;

constexpr uint32_t kPart = 1024;     // tokens of a part
constexpr uint32_t kMaxParts = (LP_MAX_SAMPLE_VOCAB + 7 + kPart - 1) / kPart;
constexpr uint32_t kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kScanResident = 4, kDrawResident = 3;  // CTAs per SM
constexpr uint32_t kMaxCluster = 8;
constexpr uint32_t kList = 1024;     // tokens that are ranked
constexpr uint32_t kRanks = kList / kThreads;  // of a thread
constexpr uint32_t kListedTop = kList * 3 / 8;  // top-k up to which what can be kept is listed at once: the bound lets two to three times as many pass
constexpr uint32_t kOrdered = 8 * kThreads;  // rows that a CTA puts in order
constexpr uint32_t kDrawnByList = 128;  // tokens up to which the draw is made from the list
constexpr uint32_t kBins = 32;
constexpr uint32_t kBound = 512;
constexpr uint32_t kTable = 256;
constexpr uint32_t kLowest = 0x00800000u;  // ordered() of the lowest finite value
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kUnit = 8796093022208.f;  // 2^43: weights as integers, the largest one is about that
// What a histogram's sums of f32 weights can be off by, of the whole: 2^-18 and less (an exponent of 40
// rounded to 2^-19, times ln 2, and the sums of some hundred).
constexpr float kSlack = 1.f / 65536.f;

// What the first kernel tells of a part.
struct Part {
    uint32_t top;                // ordered() of its largest value (a NaN's is above all)
    union {
        uint32_t lanes[3];       // keys that the 4, 16 and 32 largest of its lanes' largest reach (top-k)
        struct {
            uint32_t unused, sum_low, sum_high;  // its weights, relative to its own largest value
        };
    };
};
static_assert(sizeof(Part) == 16, "one access");

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
    Part* told;      // [T][parts]
    uint32_t* order; // [T]: the rows in the order in which they are drawn, or NULL: the last one first
    uint64_t stride;
    uint32_t T, V, B, parts;
};

// A value's bits in the order of the values (both zeros were made one before).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// The coarse bins of the values: sixteen to an octave from 2^-3 to 2^13 on both sides of 0.
__device__ __forceinline__ uint32_t bound_bin(float x) {
    const uint32_t a = (__float_as_uint(x) & 0x7FFFFFFFu) >> 19;
    const uint32_t i = min(max(a, 1984u) - 1984u, 255u);
    return x < 0.f ? 255 - i : 256 + i;
}
__device__ __forceinline__ uint32_t bound_edge(uint32_t bin) {  // ordered() of the least value in it
    if (bin > 256) return ordered(__uint_as_float((bin - 256 + 1984) << 19));
    if (bin == 256) return ordered(0.f);
    return bin == 0 ? kLowest : ordered(-__uint_as_float(((1985 + 255 - bin) << 19) - 1));
}

// What a row is drawn with.
struct Setting {
    uint32_t ok;           // 0: no token
    float tau, chi, clo;   // chi + clo = log2(e) / tau
    float top_p, min_p, u;
    uint32_t k;            // 0: off
    __device__ __forceinline__ bool weighed() const { return ok && !k && (top_p < 1.f || min_p == 0.f); }  // all weights are needed
};

struct Cut {
    uint32_t key, id;      // kept: a larger key, or this one with an id up to this
    uint32_t again;        // the search goes on among keys above `above`, for the weight `target`
    uint32_t above;
    uint64_t target;
};

struct Range {             // keys among which the cut is
    uint32_t lo, hi;
    uint32_t end;          // the least key of the first bin
    uint32_t above_count;  // how many lie above them, in the histogram's range (by count)
    uint32_t none;         // by count: there are not as many
    uint32_t fits;         // no more than a list holds
    uint32_t all_fit;      // even with what lies above them
    uint32_t narrowed, more;  // than before; than one bin
    float above, slip;     // by weight: what lies above them, and what that can be off by
};

struct Shared {
    union {
        uint64_t list[kList];    // key << 32 | ~id; the ranked tokens' weights
        uint32_t bound[kBound];  // (before the list)
    };
    uint64_t stage[kList];       // a CTA's part of the list; the ranked list
    float bin_sum[kMaxCluster][kBins];
    float2 table[kTable];
    uint64_t part_sum[kMaxParts];  // kept weights (or numbers) of the parts
    uint32_t part_top[kMaxParts];
    uint64_t scan[kWarps];
    Setting set;
    Cut cut;
    Range range;
    uint32_t edge[3];
    uint32_t listed, staged, place, top;
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
__device__ __forceinline__ uint32_t sharing(uint32_t n) { return n <= kThreads / 8 ? 3 : n <= kThreads / 4 ? 2 : n <= kThreads / 2 ? 1 : 0; }
// n different keys (n <= kList) of `from` in descending order, to `to`. They are put into a bucket a
// thread by value, and ranked among those of their bucket (300 keys: 0.9 us; counted among all, 7).
// `scratch`: kList keys and kThreads + 1 words.
__device__ __forceinline__ void sort_list(const uint64_t* from, uint64_t* to, uint32_t n, uint64_t* scratch, uint64_t* scan) {
    uint64_t* const by_bucket = scratch;
    uint32_t* const count = reinterpret_cast<uint32_t*>(scratch + kList);
    const uint32_t t = threadIdx.x;
    uint64_t key[kRanks];
    uint32_t low = kAll, high = 0;
#pragma unroll
    for (uint32_t i = 0; i < kRanks; ++i) {
        const uint32_t at = t + i * kThreads;
        key[i] = at < n ? from[at] : 0;
        if (at < n) {
            low = min(low, (uint32_t)(key[i] >> 32));
            high = max(high, (uint32_t)(key[i] >> 32));
        }
    }
    low = __reduce_min_sync(0xFFFFFFFFu, low);
    high = __reduce_max_sync(0xFFFFFFFFu, high);
    uint32_t* const ends = reinterpret_cast<uint32_t*>(scan);
    if ((t & 31) == 0) {
        ends[t / 32] = low;
        ends[kWarps + t / 32] = high;
    }
    count[t] = 0;
    __syncthreads();
#pragma unroll
    for (uint32_t k = 0; k < kWarps; ++k) {
        low = min(low, ends[k]);
        high = max(high, ends[kWarps + k]);
    }
    const float top = unordered(high), per_bucket = ((float)kThreads - 0.01f) / fminf(top - unordered(low), 3e38f);
    uint32_t bucket[kRanks], place[kRanks];
#pragma unroll
    for (uint32_t i = 0; i < kRanks; ++i) {
        bucket[i] = min((uint32_t)((top - unordered((uint32_t)(key[i] >> 32))) * per_bucket), kThreads - 1);  // (one value: 0)
        place[i] = t + i * kThreads < n ? atomicAdd(&count[bucket[i]], 1) : 0;
    }
    __syncthreads();
    const uint32_t own = count[t];
    uint64_t all;
    const uint32_t start = (uint32_t)block_scan(own, scan, &all) - own;
    __syncthreads();
    count[t] = start;
    if (t == 0) count[kThreads] = n;
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < kRanks; ++i)
        if (t + i * kThreads < n) by_bucket[count[bucket[i]] + place[i]] = key[i];
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < kRanks; ++i) {
        if (t + i * kThreads >= n) continue;
        const uint32_t begin = count[bucket[i]], end = count[bucket[i] + 1];
        uint32_t rank = begin;
        for (uint32_t j = begin; j < end; ++j) rank += by_bucket[j] > key[i];
        to[rank] = key[i];
    }
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

// A part of a row, in units of aligned vectors: element i of the row is number i + before, a part is
// 1024 numbers, and what lies outside the row is -inf.
template <typename T>
struct Row {
    static constexpr uint32_t VEC = Vec<T>::kElems, kVecs = kPart / 32 / VEC;  // vectors of a lane
    const T* x;
    uint32_t before, V;
    __device__ __forceinline__ Row(const SampleParams& p, uint32_t row)
        : x(static_cast<const T*>(p.logits) + (uint64_t)row * p.stride),
          before((uint32_t)(reinterpret_cast<uintptr_t>(x) / sizeof(T)) % VEC), V(p.V) {}
    __device__ __forceinline__ T element(uint32_t number) const {
        return number >= before && number < V + before ? x[number - before] : from_f32<T>(-__builtin_huge_valf());
    }
    // vector j of a lane: elements (32 j + lane) VEC + 0, 1, ... of the part
    __device__ __forceinline__ void load(uint32_t part, uint4 (&w)[kVecs]) const {
        const uint32_t lane = threadIdx.x & 31, begin = part * kPart;
        if (begin >= before && begin + kPart <= V + before) {
            const uint4* from = reinterpret_cast<const uint4*>(x + (begin - before)) + lane;
#pragma unroll
            for (uint32_t j = 0; j < kVecs; ++j) w[j] = from[32 * j];
        } else {
#pragma unroll
            for (uint32_t j = 0; j < kVecs; ++j) {
                T e[VEC];
#pragma unroll
                for (uint32_t i = 0; i < VEC; ++i) e[i] = element(begin + (32 * j + lane) * VEC + i);
                memcpy(&w[j], e, 16);
            }
        }
    }
};

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

__device__ __forceinline__ uint64_t warp_total(uint64_t v) {
#pragma unroll
    for (int k = 16; k > 0; k /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, k);
    return v;
}

// The rows in the order in which they are drawn, kOrdered at a time by a CTA: those that take longest first, and
// of a kind those that were read last. The last rows to be drawn are then short ones, and CTAs that run at a time do
// the same. (Rows of every kind, without and with: 256 of 128256 109 and 92 us, 2000 of 16000 166 and 123; where all are
// of one kind it costs 0.5 us, 2 to 4 of thousands of short rows. 1024 rows a CTA: 131 us of the 2000.)
__device__ __forceinline__ void order_rows(const SampleParams& p, uint64_t* scan) {
    constexpr uint32_t kEach = kOrdered / kThreads;
    const uint32_t base = blockIdx.x * kOrdered, each = (min(p.T - base, kOrdered) + kThreads - 1) / kThreads;
    const uint32_t begin = base + threadIdx.x * each;
    uint32_t kind[kEach];  // 0: longest; of row T - 1 - i, in units of bits
    uint64_t own = 0, all;
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
        if (i >= each || begin + i >= p.T) continue;
        const uint32_t row = p.T - 1 - (begin + i);
        int b = (int)min(row, p.B - 1);  // (request `row`, where every one has one row)
        if (p.row_offsets && !(p.row_offsets[b] <= row && row < p.row_offsets[b + 1])) b = max(request_of(p.row_offsets, p.B, row), 0);
        const bool best = p.temperature && p.temperature[b] == 0.f, cut = p.top_p && p.top_p[b] < 1.f, low = p.min_p && p.min_p[b] > 0.f;
        const int k = best ? 1 : p.top_k ? p.top_k[b] : 0;
        const bool listed = k > 0 && (uint32_t)k < p.V;
        kind[i] = listed ? ((uint32_t)k > kListedTop ? 0 : (uint32_t)k > kDrawnByList ? 16 : k > 1 ? 32 : 48)
                         : cut ? 0 : low ? 32 : 48;  // 0: histograms
        own += 1ull << kind[i];
    }
    uint64_t place = block_scan(own, scan, &all) - own;
    place += all << 16;  // (of a kind: after all of those before it)
    place += all << 32;
    place += all << 48;
#pragma unroll
    for (uint32_t i = 0; i < kEach; ++i) {
        if (i >= each || begin + i >= p.T) continue;
        p.order[base + (uint32_t)(place >> kind[i] & 0xFFFFu)] = p.T - 1 - (begin + i);
        place += 1ull << kind[i];
    }
}

// ---------------------------------------------------------------- the first kernel: a part a warp

template <typename T>
__global__ void __launch_bounds__(kThreads, kScanResident) k_sample_scan(const SampleParams p) {
    constexpr uint32_t VEC = Row<T>::VEC, kVecs = Row<T>::kVecs;
    __shared__ float2 table[kTable];
    const uint32_t t = threadIdx.x, lane = t & 31;
    table[t] = g_table.at[t];
    __syncthreads();
    pdl_wait();
    pdl_trigger();  // (the second kernel waits for this one before it reads what it tells)
    const uint32_t ordering = p.order ? (p.T + kOrdered - 1) / kOrdered : 0;  // CTAs that do this
    if (blockIdx.x < ordering) {
        __shared__ uint64_t scan[kWarps];
        order_rows(p, scan);
        return;
    }
    const uint32_t at = (blockIdx.x - ordering) * kWarps + (t >> 5), row = at / p.parts, part = at - row * p.parts;
    if (row >= p.T) return;
    const Row<T> r(p, row);
    uint4 w[kVecs];
    r.load(part, w);
    const Setting set = setting_of(p, row, false);
    float top = -__builtin_huge_valf();
#pragma unroll
    for (uint32_t j = 0; j < kVecs; ++j) {
        float f[VEC];
        widen(w[j], f, T());
#pragma unroll
        for (uint32_t i = 0; i < VEC; i += 2) top = max_nan(top, f[i], f[i + 1]);
    }
    Part told = {};
    const uint32_t mine = ordered(top);
    told.top = __reduce_max_sync(0xFFFFFFFFu, mine);  // (max.NaN's NaN is positive)
    if (set.k) {
        // the lanes' largest, sorted
        uint32_t v = mine;
#pragma unroll
        for (uint32_t k = 2; k <= 32; k *= 2)
#pragma unroll
            for (uint32_t j = k / 2; j > 0; j /= 2) {
                const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, v, j);
                v = ((lane & j) == 0) == ((lane & k) == 0) ? max(v, o) : min(v, o);
            }
        told.lanes[0] = __shfl_sync(0xFFFFFFFFu, v, 3);
        told.lanes[1] = __shfl_sync(0xFFFFFFFFu, v, 15);
        told.lanes[2] = __shfl_sync(0xFFFFFFFFu, v, 31);
    } else if (set.weighed() && told.top >= kLowest && told.top < ordered(__builtin_huge_valf())) {
        const Scale scale = scale_of(unordered(told.top), set);
        Weight s = {0.f, 0.f};
#pragma unroll
        for (uint32_t j = 0; j < kVecs; ++j) {
            float f[VEC];
            widen(w[j], f, T());
            float high = f[0];
#pragma unroll
            for (uint32_t i = 1; i < VEC; ++i) high = fmaxf(high, f[i]);
            if (!__any_sync(0xFFFFFFFFu, high >= scale.low)) continue;
#pragma unroll
            for (uint32_t i = 0; i < VEC; ++i) add(s, weigh(f[i], scale, table));
        }
        const uint64_t sum = warp_total(fixed(s));
        told.sum_low = (uint32_t)sum;
        told.sum_high = (uint32_t)(sum >> 32);
    }
    if (lane == 0) *reinterpret_cast<uint4*>(&p.told[at]) = *reinterpret_cast<const uint4*>(&told);
}

// ---------------------------------------------------------------- the second kernel: a row a cluster

template <typename T>
__global__ void __launch_bounds__(kThreads, kDrawResident) k_sample_draw(const SampleParams p) {
    constexpr uint32_t VEC = Row<T>::VEC, kVecs = Row<T>::kVecs;
    constexpr float kInf = __builtin_huge_valf();
    __shared__ Shared sh;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    unsigned char (*const buffers)[4 * kPart] = reinterpret_cast<unsigned char (*)[4 * kPart]>(smem_raw);  // of a warp: a part, or 32 sums a lane
    T* const buffer = reinterpret_cast<T*>(buffers[threadIdx.x >> 5]);
    const cg::cluster_group cluster = cg::this_cluster();
    const uint32_t C = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5, parts = p.parts;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (waited for before others' memory is written to)
    sh.table[t] = g_table.at[t];
    for (uint32_t i = t; i < kBound; i += kThreads) sh.bound[i] = 0;
    if (t == 0) sh.staged = sh.listed = sh.top = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    // (the rows that the first kernel read last come first: they are in L2)
    const uint32_t row = p.order ? min(__ldcg(p.order + blockIdx.x / C), p.T - 1) : p.T - 1 - blockIdx.x / C;
    const Row<T> r(p, row);
    const auto id_of = [&](uint32_t part, uint32_t element) { return part * kPart + element - r.before; };

    // ---- 1. what the parts tell
    const uint4* told = reinterpret_cast<const uint4*>(p.told + (uint64_t)row * parts);
    uint4 info[(kMaxParts + kThreads - 1) / kThreads];
    uint32_t top = 0;
#pragma unroll
    for (uint32_t i = 0; i < (kMaxParts + kThreads - 1) / kThreads; ++i) {
        info[i] = t + i * kThreads < parts ? __ldcg(told + t + i * kThreads) : make_uint4(0, 0, 0, 0);
        top = max(top, info[i].x);
    }
    if (t == 0) sh.set = setting_of(p, row, rank == 0);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) atomicMax(&sh.top, top);
    __syncthreads();
    const Setting set = sh.set;
    uint32_t hi = sh.top, lo = kLowest;  // keys below `lo` are not kept
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (!set.ok || hi < kLowest || hi >= ordered(kInf)) {
        if (rank == 0 && t == 0) {
            if (set.ok) flag(p.status, LP_ERR_LOGITS);
            p.out[row] = kAll;
            if (p.out_logprob) p.out_logprob[row] = __uint_as_float(0x7FC00000u);
        }
        return;
    }
    // (without a filter, and for the best token, the first CTA is enough)
    if (rank != 0 && (set.k == 1 || (!set.k && set.top_p == 1.f && set.min_p == 0.f))) return;
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
    // The elements of the parts that hold values of [from, ...], for the warps of the cluster in turn:
    // body(part, values of a lane's vectors).
    const auto for_parts = [&](float from, auto body) {
        const uint32_t key = ordered(from);
        for (uint32_t part = rank * kWarps + warp; part < parts; part += C * kWarps) {
            if (sh.part_top[part] < key) continue;
            uint4 w[kVecs];
            r.load(part, w);
            body(part, w);
        }
    };
    // Visits the elements with values of `from` or more, two at a time: body(part, element, element or kAll,
    // value, value), then after(part). Lanes take them out of masks of 32, so that few cost little.
    const auto visit = [&](float from, auto body, auto after) {
        for_parts(from, [&](uint32_t part, const uint4 (&w)[kVecs]) {
            uint32_t take = 0;
            __syncwarp();
#pragma unroll
            for (uint32_t j = 0; j < kVecs; ++j) {
                float f[VEC];
                widen(w[j], f, T());
                float high = f[0];
#pragma unroll
                for (uint32_t i = 1; i < VEC; ++i) high = fmaxf(high, f[i]);
                if (!__any_sync(0xFFFFFFFFu, high >= from)) continue;
                reinterpret_cast<uint4*>(buffer)[j * 32 + lane] = w[j];
#pragma unroll
                for (uint32_t i = 0; i < VEC; ++i)
                    if (f[i] >= from) take |= 1u << (j * VEC + i);
            }
            __syncwarp();
            const auto next = [&] {  // (without branches)
                const uint32_t b = __ffs(take) - 1, e = (b / VEC * 32 + lane) * VEC + b % VEC;
                const bool some = take != 0;
                take &= take - 1;
                return some ? e : kAll;
            };
            while (__any_sync(0xFFFFFFFFu, take)) {
                const uint32_t e0 = next(), e1 = next();
                const float x0 = to_f32(buffer[min(e0, kPart - 1)]) + 0.f, x1 = to_f32(buffer[min(e1, kPart - 1)]) + 0.f;
                const float f0 = e0 == kAll ? -kInf : x0, f1 = e1 == kAll ? -kInf : x1;
                body(part, e0, e1, f0, f1);
            }
            after(part);
        });
    };
    const auto no_more = [](uint32_t) {};
    // A part's sum, told to all CTAs; those of parts that are not visited stay 0.
    const auto clear_sums = [&] {
        for (uint32_t i = t; i < parts; i += kThreads) sh.part_sum[i] = 0;
    };
    const auto tell = [&](uint32_t part, uint64_t sum) {
        if (lane < C) cluster.map_shared_rank(&sh, lane)->part_sum[part] = sum;
    };
    const auto told_total = [&] {
        uint64_t sum = 0;
        for (uint32_t i = lane; i < parts; i += 32) sum += sh.part_sum[i];
        return warp_total(sum);
    };
    // The sum of the weights of values of at least `from`; begins and ends with a barrier of the cluster.
    const auto sum_from = [&](float from) {
        cluster.sync();  // (the sums told before have been read)
        clear_sums();
        cluster.sync();
        Weight s = {0.f, 0.f};
        visit(from, [&](uint32_t, uint32_t, uint32_t, float f0, float f1) {
            add(s, weight_of(f0));
            add(s, weight_of(f1));
        }, [&](uint32_t part) {
            tell(part, warp_total(fixed(s)));
            s = {0.f, 0.f};
        });
        cluster.sync();
        return told_total();
    };

    // ---- 2. the parts' largest; their weights, relative to the row's largest; a bound for the k-th value
#pragma unroll
    for (uint32_t i = 0; i < (kMaxParts + kThreads - 1) / kThreads; ++i) {
        const uint32_t part = t + i * kThreads;
        if (part >= parts) continue;
        sh.part_top[part] = info[i].x;
        uint64_t sum = 0;
        if (set.weighed() && info[i].x >= ordered(scale.low)) {  // (one at least of its tokens can be drawn)
            // sums are in units of 2^(x (chi + clo) - shift) each: shift of the part, and of the row
            const Scale own = scale_of(unordered(info[i].x), set);
            const bool far = own.base != 0.f || scale.base != 0.f;
            double factor;
            if (far) {
                const double c = (double)set.chi + (double)set.clo;
                const auto origin = [&](const Scale& q) { return q.base != 0.f ? (double)q.base * c : 49152.0 - (double)q.magic; };
                factor = exp2(origin(own) - origin(scale));
            } else {
                const int k = (int)((scale.magic - own.magic) * 256.f);  // shift of the part less that of the row
                const float2 e = sh.table[k & (kTable - 1)];
                factor = k < -126 * 256 ? 0.0 : ((double)e.x + (double)e.y) * (double)__uint_as_float((uint32_t)((k >> 8) + 127) << 23);
            }
            sum = __double2ull_rn((double)((uint64_t)info[i].w << 32 | info[i].z) * factor);
        }
        sh.part_sum[part] = sum;
        if (set.k && info[i].x >= kLowest) {
            // one value of `x`, three more of `y`, twelve of `z` and sixteen of `w` at least
            const uint32_t key[4] = {info[i].x, info[i].y, info[i].z, info[i].w}, more[4] = {1, 3, 12, 16};
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
                if (key[k] >= kLowest) atomicAdd(&sh.bound[bound_bin(unordered(key[k]))], more[k]);
        }
    }
    __syncthreads();

    Shared* lead = cluster.map_shared_rank(&sh, 0);
    Cut cut = {least, kAll, 0, 0, 0};
    const auto kept = [&](float f, uint32_t id) {
        const uint32_t key = ordered(f);
        return (key > cut.key) | ((key == cut.key) & (id <= cut.id));
    };
    const auto add_to_part = [&](uint64_t entry, uint64_t w) {  // of a ranked token
        if (w)
            atomicAdd(reinterpret_cast<unsigned long long*>(&sh.part_sum[(~(uint32_t)entry + r.before) / kPart]), (unsigned long long)w);
    };
    // The draw, by one CTA, from the parts' sums of kept weights: the part in which u Z falls, and in it
    // the token, four neighbours to a thread.
    const auto finish = [&] {
        const uint32_t each = (parts + 31) / 32;
        uint64_t own = 0;
        for (uint32_t i = lane * each; i < min(lane * each + each, parts); ++i) own += sh.part_sum[i];
        const uint64_t upto = warp_scan(own), z = __shfl_sync(0xFFFFFFFFu, upto, 31);
        bool exact;
        const uint64_t want = part_of(set.u, z, &exact);
        uint64_t below = upto - own;
        uint32_t part = kAll;
        if (below <= want && want < upto)
            for (uint32_t i = lane * each; i < min(lane * each + each, parts); ++i) {
                if (want < below + sh.part_sum[i]) {
                    part = i;
                    break;
                }
                below += sh.part_sum[i];
            }
        const int src = __ffs(__ballot_sync(0xFFFFFFFFu, part != kAll)) - 1;  // (one lane: want < z)
        part = __shfl_sync(0xFFFFFFFFu, part, src);
        below = __shfl_sync(0xFFFFFFFFu, below, src);
        float f[kPart / kThreads];
        uint64_t w[kPart / kThreads], here = 0, all;
#pragma unroll
        for (uint32_t i = 0; i < kPart / kThreads; ++i) {
            const uint32_t e = t * (kPart / kThreads) + i;
            f[i] = to_f32(r.element(part * kPart + e)) + 0.f;
            const Weight q = weight_of(kept(f[i], id_of(part, e)) ? f[i] : -kInf);
            w[i] = enough(q) ? fixed(q) : 0;
            here += w[i];
        }
        uint64_t under = block_scan(here, sh.scan, &all) - here;
        // (these sums are rounded another way than the part's: at its very end the last kept is meant)
        const uint64_t left = min(want - below, all - 1);
#pragma unroll
        for (uint32_t i = 0; i < kPart / kThreads; ++i) {
            if (under <= left && left < under + w[i]) token_is(id_of(part, t * (kPart / kThreads) + i), f[i], z);
            under += w[i];
        }
    };
    if (set.k == 1) {
        // the first token that has the largest value
        uint32_t first = kAll;
        for (uint32_t i = lane; i < parts; i += 32)
            if (sh.part_top[i] == hi) first = min(first, i);
        first = __reduce_min_sync(0xFFFFFFFFu, first);
        uint32_t id = kAll;
#pragma unroll
        for (uint32_t i = 0; i < kPart / kThreads; ++i) {
            const uint32_t e = t + i * kThreads;
            if (to_f32(r.element(first * kPart + e)) + 0.f == m) id = min(id, id_of(first, e));
        }
        id = __reduce_min_sync(0xFFFFFFFFu, id);
        if (lane == 0) sh.scan[warp] = id;
        __syncthreads();
        if (t == 0) {
            for (uint32_t k = 1; k < kWarps; ++k) id = min(id, (uint32_t)sh.scan[k]);
            token_is(id, m, fixed(most));
        }
        return;
    }
    if (!set.k && set.top_p == 1.f && set.min_p == 0.f) {
        finish();
        return;
    }
    // Tokens into the CTA's part of the list, and the parts into the first CTA's, which ends with a barrier of
    // the cluster.
    const auto stage = [&](uint32_t part, uint32_t e0, uint32_t e1, float f0, float f1) {
        const auto one = [&](uint32_t e, float f) {
            const uint32_t take = __ballot_sync(0xFFFFFFFFu, e != kAll);
            if (!take) return;
            uint32_t at = 0;
            if (lane == 0) at = atomicAdd(&sh.staged, __popc(take));
            at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(take & ((1u << lane) - 1));
            if (e != kAll && at < kList) sh.stage[at] = (uint64_t)ordered(f) << 32 | (uint32_t)~id_of(part, e);
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

    if (set.k || set.top_p < 1.f) {
        uint64_t target = set.k;
        bool by_count = set.k != 0, few = set.k <= kListedTop;
        if (by_count) {
            // from the top: lane 0 has the largest bins
            if (warp == 0) {
                uint32_t n[kBound / 32], sum = 0, bin = kAll;
#pragma unroll
                for (uint32_t i = 0; i < kBound / 32; ++i) sum += n[i] = sh.bound[kBound - 1 - (lane * (kBound / 32) + i)];
                uint32_t have = warp_scan(sum) - sum;
#pragma unroll
                for (uint32_t i = 0; i < kBound / 32; ++i) {
                    if (have < set.k && have + n[i] >= set.k) bin = kBound - 1 - (lane * (kBound / 32) + i);
                    have += n[i];
                }
                bin = __reduce_min_sync(0xFFFFFFFFu, bin);
                if (lane == 0) sh.place = bin == kAll ? kLowest : bound_edge(bin);
            }
            __syncthreads();
            lo = sh.place;
            cluster.sync();  // (the bins: the list takes their place)
        } else {
            const uint64_t z = told_total();
            target = reached_at(set.top_p, z);
            const float sum = (float)z / kUnit;
            // kept tokens weigh (1 - p) Z / V at least (with room for the roundings here)
            const float f = m + set.tau * (__logf((1.f - set.top_p) * sum / (float)p.V) - 0.02f) - fabsf(m) * 1e-6f;
            lo = f > -3e38f ? min(max(ordered(f + 0.f), kLowest), hi) : kLowest;
            // Tokens are few where not nearly every part has one. (Looking for them in vain costs 12 us of a row's 50.)
            uint32_t with = 0;
            for (uint32_t i = t; i < parts; i += kThreads) with += sh.part_top[i] >= lo;
            with = __reduce_add_sync(0xFFFFFFFFu, with);
            __syncthreads();
            if (lane == 0) sh.scan[warp] = with;
            __syncthreads();
            with = 0;
            for (uint32_t k = 0; k < kWarps; ++k) with += (uint32_t)sh.scan[k];
            few = p.V <= kList || 20 * with < 19 * parts;
        }
        // ---- 4. the value at which the target is reached, by histograms over [lo, hi]
        bool found = false, read = false;  // whether others may still read the tables and the list
        uint32_t above_count = 0;        // by count: of the keys above hi
        float rough = 0.f, slip = 0.f;   // by weight: their weight, and what that can be off by
        for (int n_hist = 0; n_hist < 64 && !found; ++n_hist) {  // (a bound only: each cuts the range)
            // ---- 3. all that can be kept in one list? (at once, or when a histogram has told so)
            if (few) {
                few = false;
                read = true;
                visit(unordered(lo), stage, no_more);
                send_list();
                const uint32_t n = lead->listed;
                if (n <= kList) {
                    // the first CTA does the rest; the others have read its count, and no one reads theirs
                    if (rank != 0) {
                        asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
                        return;
                    }
                    sort_list(sh.list, sh.stage, n, reinterpret_cast<uint64_t*>(smem_raw), sh.scan);
                    uint64_t w[kRanks], all, kept_all, sum = 0;
                    bool fine[kRanks];
#pragma unroll
                    for (uint32_t i = 0; i < kRanks; ++i) {
                        const uint32_t at = kRanks * t + i;
                        const Weight q = weight_of(at < n && (!set.k || at < set.k) ? unordered((uint32_t)(sh.stage[at] >> 32)) : -kInf);
                        w[i] = fixed(q);
                        fine[i] = w[i] && enough(q);
                        sum += w[i];
                    }
                    uint64_t below = block_scan(sum, sh.scan, &all) - sum;
                    if (by_count) target = set.top_p < 1.f ? reached_at(set.top_p, all) : ~0ull;
                    uint32_t keep = 0;
#pragma unroll
                    for (uint32_t i = 0; i < kRanks; ++i) {
                        keep += fine[i] && below < target;
                        below += w[i];
                        if (kRanks * t + i < n) sh.list[kRanks * t + i] = w[i];  // (the list is in `stage` now)
                    }
                    (void)block_scan(keep, sh.scan, &kept_all);
                    const uint32_t n_kept = (uint32_t)kept_all;
                    if (n_kept > kDrawnByList) {
                        // by the parts' sums, as where there is no list
                        const uint64_t least_kept = sh.stage[n_kept - 1];
                        cut = {(uint32_t)(least_kept >> 32), ~(uint32_t)least_kept, 0, 0, 0};
                        clear_sums();
                        __syncthreads();
#pragma unroll
                        for (uint32_t i = 0; i < kRanks; ++i)
                            if (kRanks * t + i < n_kept) add_to_part(sh.stage[kRanks * t + i], w[i]);
                        __syncthreads();
                        finish();
                    } else {
                        // The kept in the order of their ids: what lies below each.
                        const uint32_t shift = sharing(n_kept), share = 1u << shift, at = t >> shift;
                        const uint64_t entry = at < n_kept ? sh.stage[at] : 0;
                        const uint32_t not_id = (uint32_t)entry;
                        uint64_t under = 0, z = 0;
#pragma unroll 8
                        for (uint32_t j = t & (share - 1); j < n_kept; j += share) {
                            const uint64_t wj = sh.list[j];
                            under += (uint32_t)sh.stage[j] > not_id ? wj : 0;
                            z += wj;
                        }
                        for (uint32_t k = 1; k < share; k *= 2) {
                            under += __shfl_xor_sync(0xFFFFFFFFu, under, k);
                            z += __shfl_xor_sync(0xFFFFFFFFu, z, k);
                        }
                        bool exact;
                        const uint64_t want = part_of(set.u, z, &exact);
                        if (at < n_kept && (t & (share - 1)) == 0 && under <= want && want < under + sh.list[at])
                            token_is(~not_id, unordered((uint32_t)(entry >> 32)), z);
                    }
                    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
                    return;
                }
            }
            // 31 bins of equal width, and from the second time on (or where that is all of f32) of equally many
            // keys: what is left is within an octave mostly, and a cut at 0 would be neared 32-fold at a time.
            // What lies outside has a bin of its own, the last. (Below `lo` some may be in the bin of `lo`.)
            const float from = unordered(lo), to = unordered(hi), per_bin = 30.49f / (to - from);
            const bool even = n_hist == 0 && to - from < 1e38f && to - from > 1e-30f && !(by_count && lo == kLowest);
            uint32_t shift = 27 - min(__clz(hi - lo | 1), 27);
            shift += (hi - lo) >> shift >= kBins - 1;
            const auto bin_of = [&](float f, auto equal_width) {  // (decreasing in f)
                // (equal width: `to` is the row's largest; an ulp of 2^23 is 1)
                if constexpr (decltype(equal_width)::value) return min(__float_as_uint(fmaf(to - f, per_bin, 8388608.f)) - 0x4B000000u, kBins - 1);
                else return min((hi - ordered(f)) >> shift, kBins - 1);
            };
            const auto bin_at = [&](float f) { return even ? bin_of(f, std::true_type()) : bin_of(f, std::false_type()); };
            if (read) cluster.sync(); else __syncthreads();
            read = true;
            clear_sums();
            if (t == 0) sh.listed = sh.staged = 0;
            {
                // A lane adds to sums of its own (bin by lane: each in the lane's bank), without atomics, which
                // take two clocks a lane: 27000 tokens that can be kept, 13500 clocks of eight CTAs with them.
                // (by count: 2^0; no branches below, which cost this loop as much as all the rest)
                const float chi = by_count ? 0.f : -scale.chi, at_to = by_count ? 0.f : fmaf(to - scale.base, scale.chi, scale.magic - 49152.f);
                float* const sums = reinterpret_cast<float*>(buffers[warp]) + lane;
#pragma unroll
                for (uint32_t i = 0; i < kBins / 4; ++i) reinterpret_cast<uint4*>(buffers[warp])[i * 32 + lane] = make_uint4(0, 0, 0, 0);
                __syncwarp();
                const auto fill = [&](auto equal_width) {
                    for_parts(from, [&](uint32_t, const uint4 (&w)[kVecs]) {
#pragma unroll
                        for (uint32_t j = 0; j < kVecs; ++j) {
                            float f[VEC];
                            widen(w[j], f, T());
                            float high = f[0];
#pragma unroll
                            for (uint32_t i = 1; i < VEC; ++i) high = fmaxf(high, f[i]);
                            if (!__any_sync(0xFFFFFFFFu, high >= from)) continue;
#pragma unroll
                            for (uint32_t i = 0; i < VEC; ++i) {
                                float e;
                                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(to - f[i], chi, at_to)));
                                // (-inf has weight 0, but counts as 1)
                                if constexpr (!decltype(equal_width)::value) e = f[i] >= from ? e : 0.f;
                                sums[bin_of(f[i], equal_width) * 32] += e;
                            }
                        }
                    });
                };
                if (even) fill(std::true_type()); else fill(std::false_type());
                __syncthreads();
                // the CTA's, four bins a warp, to the first CTA
#pragma unroll
                for (uint32_t b = 0; b < kBins / kWarps; ++b) {
                    const uint32_t bin = warp * (kBins / kWarps) + b;
                    float sum = 0.f;
#pragma unroll
                    for (uint32_t k = 0; k < kWarps; ++k) sum += reinterpret_cast<const float*>(buffers[k])[bin * 32 + lane];
#pragma unroll
                    for (int k = 16; k > 0; k /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
                    if (lane == 0) lead->bin_sum[rank][bin] = sum;
                }
            }
            cluster.sync();
            // The first CTA finds the bins in which the target can be reached.
            if (rank == 0) {
                float own = 0.f;
                for (uint32_t k = 0; k < C; ++k) own += sh.bin_sum[k][lane];
                if (lane == kBins - 1) own = 0.f;  // (what lies outside)
                float upto = own;
#pragma unroll
                for (int k = 1; k < 32; k *= 2) {
                    const float o = __shfl_up_sync(0xFFFFFFFFu, upto, k);
                    if (lane >= k) upto += o;
                }
                // (numbers are exact: fewer than 2^24)
                const float aim = by_count ? (float)((uint32_t)target - above_count) : fmaxf((float)target / kUnit - rough, 0.f);
                const float slack = by_count ? 0.f : slip + kSlack * (__shfl_sync(0xFFFFFFFFu, upto, 31) + rough / 64.f);  // (the aim is a difference of f32)
                const uint32_t bins = min(bin_at(from), kBins - 2);
                const uint32_t can = __ballot_sync(0xFFFFFFFFu, upto >= aim - slack), must = __ballot_sync(0xFFFFFFFFu, upto >= aim + slack);
                const uint32_t last = min(must ? __ffs(must) - 1 : bins, bins), first = min(can ? __ffs(can) - 1 : last, last);
                // The least keys of bins `last`, `first` and the one above it, by a warp each: 32 keys at a time.
                if (warp < 3) {
                    const uint32_t bin = warp == 0 ? last : warp == 1 ? first : first - 1;
                    uint32_t low = lo, n = hi - lo + 1;  // it is among n keys from `low` on
                    while (n > 1) {
                        const uint32_t step = (n - 1) / 32 + 1, key = low + min(lane * step, n - 1);
                        const uint32_t below = __popc(__ballot_sync(0xFFFFFFFFu, lane * step < n && bin_at(unordered(key)) > bin));
                        if (below == 0) break;
                        const uint32_t past = (below - 1) * step + 1;  // (the next key looked at is one that has it)
                        low += past;
                        n = min(step, n - past);
                    }
                    if (lane == 0) sh.edge[warp] = low;
                }
                const float before = __shfl_sync(0xFFFFFFFFu, upto, first ? first - 1 : 0), below = first ? before : 0.f;
                const float in = __shfl_sync(0xFFFFFFFFu, upto, last) - below;
                __syncthreads();
                if (t < C) {
                    Range q;
                    q.lo = last == bins ? lo : sh.edge[0];
                    q.end = sh.edge[1];
                    q.hi = first ? sh.edge[2] - 1 : hi;
                    q.above_count = by_count ? (uint32_t)below : 0u;
                    q.none = by_count && !can;
                    // (by weight: as many as the lightest of them would make)
                    q.fits = by_count ? in <= (float)kList : in * 1.001f <= (float)kList * weight_of(unordered(q.lo)).hi;
                    // (what lies above weighs more than that each)
                    q.all_fit = by_count ? (float)above_count + below + in <= (float)kList : (rough + below + in) * 1.001f <= (float)kList * weight_of(unordered(q.lo)).hi;
                    q.narrowed = first != 0 || last != bins;
                    q.more = first != last;
                    q.above = rough + below;
                    q.slip = first ? slack : slip;
                    cluster.map_shared_rank(&sh, t)->range = q;
                }
            }
            cluster.sync();
            const Range range = sh.range;
            if (range.none) {  // all of it is kept
                if (set.top_p == 1.f) {
                    cut = {max(lo, least), kAll, 0, 0, 0};
                    found = true;
                    break;
                }
                const uint64_t z = sum_from(unordered(kLowest));
                by_count = false;
                target = reached_at(set.top_p, z);
                continue;
            }
            above_count += range.above_count;
            lo = range.lo;
            hi = range.hi;
            const bool fits = range.fits, exact = slip == 0.f && range.slip == 0.f;
            rough = range.above;
            slip = range.slip;
            few = range.all_fit;
            if (few) continue;
            // (bins of bins, for a list of all: k and p from one ranking instead of one after the other. 256 rows
            // of 128256 with both, k up to 1000: 85 -> 77 us)
            if (by_count && n_hist == 0 && set.top_p < 1.f && set.k <= kList - kList / 32 && lo != hi) continue;
            if (!fits && lo != hi) {
                if (by_count || range.narrowed || !range.more) continue;  // once more
                // A few values of many tokens, or few of the weights. On which side of the first bin's end?
                // (first, what lies above, exactly)
                const uint64_t upto_there = sum_from(unordered(exact ? range.end : hi + 1));
                if (exact && upto_there >= target) {
                    lo = range.end;
                    continue;
                }
                if (exact) hi = range.end - 1;
                rough = (float)upto_there / kUnit;
                slip = 0.f;
                continue;
            }
            // the weights above them, exactly, by part; what lies in them is listed, where it fits
            {
                Weight s = {0.f, 0.f};
                const float border = unordered(hi);
                visit(fits ? unordered(lo) : border, [&](uint32_t part, uint32_t e0, uint32_t e1, float f0, float f1) {
                    add(s, weight_of(f0 > border ? f0 : -kInf));
                    add(s, weight_of(f1 > border ? f1 : -kInf));
                    if (fits) stage(part, f0 > border ? kAll : e0, f1 > border ? kAll : e1, f0, f1);
                }, [&](uint32_t part) {
                    tell(part, warp_total(fixed(s)));
                    s = {0.f, 0.f};
                });
            }
            if (fits) send_list(); else cluster.sync();
            const uint64_t above = told_total();
            if (fits) {
                // ranked by the first CTA (by weight it ends there: the bins hold the cut for sure)
                const bool last = !by_count && set.min_p == 0.f;
                if (last && rank != 0) return;
                if (rank == 0) {
                    const uint32_t listed = min(sh.listed, kList);
                    sort_list(sh.list, sh.stage, listed, reinterpret_cast<uint64_t*>(smem_raw), sh.scan);
                    const uint32_t limit = by_count ? min(listed, (uint32_t)target - above_count) : listed;
                    uint64_t w[kRanks], own = 0, sum, kept_all;
#pragma unroll
                    for (uint32_t i = 0; i < kRanks; ++i) {
                        const uint32_t at = kRanks * t + i;
                        w[i] = fixed(weight_of(at < limit ? unordered((uint32_t)(sh.stage[at] >> 32)) : -kInf));
                        own += w[i];
                    }
                    uint64_t below = above + block_scan(own, sh.scan, &sum) - own;
                    uint64_t goal = target;
                    if (by_count) goal = set.top_p < 1.f ? reached_at(set.top_p, above + sum) : ~0ull;
                    uint32_t keep = 0;
#pragma unroll
                    for (uint32_t i = 0; i < kRanks; ++i) {
                        keep += kRanks * t + i < limit && below < goal;
                        below += w[i];
                    }
                    (void)block_scan(keep, sh.scan, &kept_all);
                    if (!by_count && kept_all == 0) kept_all = 1;  // (the margin would have been passed: cannot be)
                    cut = {kAll, 0, 1, hi, goal};  // reached among larger values
                    if (kept_all) {
                        const uint64_t least_kept = sh.stage[kept_all - 1];
                        cut = {(uint32_t)(least_kept >> 32), ~(uint32_t)least_kept, 0, 0, 0};
                        if (set.min_p == 0.f) {  // the parts' sums are complete with these
#pragma unroll
                            for (uint32_t i = 0; i < kRanks; ++i)
                                if (kRanks * t + i < kept_all) add_to_part(sh.stage[kRanks * t + i], w[i]);
                        }
                    }
                    if (last) {
                        __syncthreads();
                        finish();
                        return;
                    }
                    if (t < C) cluster.map_shared_rank(&sh, t)->cut = cut;
                }
                cluster.sync();
                cut = sh.cut;
                found = cut.again == 0;
                if (found && set.min_p == 0.f) {
                    if (rank == 0) finish();
                    return;
                }
                if (cut.again) {  // once more, by weight, among the larger values
                    by_count = false;
                    target = cut.target;
                    lo = cut.above + 1;
                    hi = ordered(m);
                    rough = slip = 0.f;
                }
            } else {
                // one value: its first `j` ids are kept
                const uint64_t one = fixed(weight_of(unordered(hi)));
                uint64_t j = by_count ? target - above_count : one ? (target - above + one - 1) / one : 1;
                if (by_count && set.top_p < 1.f) {
                    const uint64_t z = above + j * one, goal = reached_at(set.top_p, z);
                    if (goal <= above) {
                        by_count = false;
                        target = goal;
                        lo = hi + 1;
                        hi = ordered(m);
                        rough = slip = 0.f;
                        continue;
                    }
                    if (one) j = min(j, (goal - above + one - 1) / one);
                }
                // the j-th of them, counted by part in the order of the ids
                cluster.sync();  // (the sums have been read)
                clear_sums();
                cluster.sync();
                const float value = unordered(hi);
                uint32_t here = 0;
                visit(unordered(hi), [&](uint32_t, uint32_t, uint32_t, float f0, float f1) { here += (f0 == value) + (f1 == value); },
                      [&](uint32_t part) {
                          tell(part, __reduce_add_sync(0xFFFFFFFFu, here));
                          here = 0;
                      });
                cluster.sync();
                if (rank == 0 && warp == 0) {
                    // the part that has it, and its place there
                    uint64_t left = j;
                    uint32_t part = 0;
                    while (part < parts && left > sh.part_sum[part]) left -= sh.part_sum[part++];
                    uint32_t id = kAll;
                    for (uint32_t e0 = 0; part < parts && e0 < kPart; e0 += 32) {
                        const bool is = to_f32(r.element(part * kPart + e0 + lane)) + 0.f == unordered(hi);
                        const uint32_t who = __ballot_sync(0xFFFFFFFFu, is), n = __popc(who);
                        if (left > n) {
                            left -= n;
                            continue;
                        }
                        if (is && __popc(who & ((2u << lane) - 1)) == (uint32_t)left) id = id_of(part, e0 + lane);
                        break;
                    }
                    id = __reduce_min_sync(0xFFFFFFFFu, id);
                    if (lane < C) cluster.map_shared_rank(&sh, lane)->cut.id = id;
                }
                cluster.sync();
                cut = {hi, sh.cut.id, 0, 0, 0};
                found = true;
            }
        }
        if (least > cut.key) cut = {least, kAll, 0, 0, 0};
    }

    // ---- 5. the kept weights by part
    cluster.sync();  // (the sums told before have been read)
    clear_sums();
    cluster.sync();
    Weight s = {0.f, 0.f};
    visit(unordered(cut.key), [&](uint32_t part, uint32_t e0, uint32_t e1, float f0, float f1) {
        const Weight a = weight_of(e0 != kAll && kept(f0, id_of(part, e0)) ? f0 : -kInf);
        const Weight b = weight_of(e1 != kAll && kept(f1, id_of(part, e1)) ? f1 : -kInf);
        if (enough(a)) add(s, a);
        if (enough(b)) add(s, b);
    }, [&](uint32_t part) {
        tell(part, warp_total(fixed(s)));
        s = {0.f, 0.f};
    });
    cluster.sync();
    if (rank == 0) finish();
}

uint32_t parts_of(uint32_t V) { return (V + 7 + kPart - 1) / kPart; }  // (rows begin up to seven elements past a boundary)

template <typename T>
lp_status launch_sample(SampleParams& p, lp_stream_t stream) {
    static std::atomic<uint64_t> smem_set;
    constexpr size_t kBuffers = (size_t)kWarps * 4 * kPart;
    if (!allow_smem(reinterpret_cast<const void*>(k_sample_draw<T>), kBuffers, &smem_set)) return LP_ERR_CUDA;
    // CTAs of a row: two parts to a warp, eight CTAs at most; of many rows, so many that all CTAs are twice
    // what the device holds at once (256 rows of 128256, all with top-p: 8 CTAs 221 us, 4 198, 2 239; one row 32, 38, 52).
    const uint32_t slots = 2 * kDrawResident * (uint32_t)sm_count();
    uint32_t c = 1;
    while (c < kMaxCluster && c * kWarps * 2 < p.parts && 2 * (uint64_t)c * p.T <= slots + slots / 4) c *= 2;
    // In order where there are more than the device holds.
    if ((uint64_t)c * p.T <= slots / 2) p.order = nullptr;
    const uint32_t ordering = p.order ? (p.T + kOrdered - 1) / kOrdered : 0;
    const uint64_t warps = (uint64_t)p.T * p.parts;
    const lp_status st = launch(k_sample_scan<T>, dim3((unsigned)((warps + kWarps - 1) / kWarps) + ordering), kThreads, 0, stream, 1, p);
    if (st != LP_OK) return st;
    return launch(k_sample_draw<T>, dim3(p.T * c), kThreads, kBuffers, stream, c, p);
}

}  // namespace

extern "C" size_t lp_head_sample_workspace_size(uint32_t T, uint32_t V) {
    return kHeaderBytes + (size_t)T * (parts_of(V) * sizeof(Part) + sizeof(uint32_t));
}

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
    if ((uint64_t)T * parts_of(V) > 0x7FFFFFFFu) return LP_ERR_SHAPE;
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < lp_head_sample_workspace_size(T, V)) return LP_ERR_WORKSPACE;
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
    p.told = reinterpret_cast<Part*>(static_cast<unsigned char*>(workspace) + kHeaderBytes);
    p.parts = parts_of(V);
    p.order = reinterpret_cast<uint32_t*>(p.told + (size_t)T * p.parts);
    p.stride = stride;
    p.T = T;
    p.V = V;
    p.B = B;
    if (dtype == LP_F32) return launch_sample<float>(p, stream);
    if (dtype == LP_BF16) return launch_sample<__nv_bfloat16>(p, stream);
    return launch_sample<__half>(p, stream);
}
