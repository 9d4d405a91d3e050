// Processing of logits before they are scored or sampled: penalties for repeated tokens,
// biases, grammar masks (include/lp_head.h).
//
// A CTA takes a slice of the vocabulary of one logits row. For the request's history it keeps a
// table in shared memory, 16 bits a token of the slice: the count in the output part and, in
// the top bit, whether the prompt holds it (adds and ors of integers, so their order does not
// matter); 32 bits, and the slice in two halves, for a request whose output part could overflow
// 15 bits. With many tokens of the slice in the table every value looks at its word while the
// slice is copied from logits to out. With few the slice is copied first, and then each
// token's word is taken out of the table (the first thread to come gets it) and its value
// corrected. Biases are added last. Long histories are sorted by slices first (k_sort_history,
// 4096 tokens a CTA, into the workspace); short ones are read by every CTA of a row.
//
// A row is read once and written once, and a vector whose mask bits are all 0 is not read; HBM
// would take 41 us for 256 rows of 128256 f32, and without lists this takes that. What costs is
// the time before the copy (who the row belongs to, its parameters, its history: reads that wait
// for each other, about 6 of a CTA's 17 us), and the copy's look at the table (8 against 4 us).
// So the slice is asked for in L2 at the very start (57 -> 41 us) and the mask read while one warp
// finds the row's request (66 -> 62 us with histories of up to 30000), the histories are sorted
// while the first CTAs begin, and four or five CTAs share an SM.
// Slices held in shared memory as values, loaded and stored by bulk copies, were measured too:
// 36000 tokens per SM at a time instead of 98000 hide less of those waits (85 us).
#include "lp_head_common.h"

namespace {

using namespace lph;

// Tokens of a slice: a 48 KB table, four CTAs per SM (256 rows of 128256 f32 with histories of up
// to 30000, 240 rows of 152064 bf16 with up to 3000: 69 and 47 us; 16384, five CTAs: 71 and 54).
constexpr uint32_t kMaxSlice = 24576;
constexpr uint32_t kMinSlice = 1024;
constexpr uint32_t kResident = 4;      // CTAs per SM
constexpr uint32_t kBatch = 4;         // vectors a thread has in flight
constexpr uint32_t kChunk = 4096;      // tokens of a history sorted together
constexpr uint32_t kSortFrom = 4096;   // mean length from which histories are sorted first
constexpr uint32_t kMaxSlices = 256;
constexpr uint32_t kOrderedWord = 32;  // of the workspace's header: 1 where history_offsets nowhere decrease

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
    uint32_t* sorted;  // [history_total], NULL: histories are not sorted
    uint32_t* bounds;  // [chunks][slices + 1]
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
// costs about ten instructions (256 rows with histories of up to 30000: 69 us instead of 62).
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
    uint32_t h0, h1, prompt; // its history, and how much of that is the prompt
    uint32_t b0, b1;         // its biases
    Penalty q;
};

// The request of row t, found by one warp: 32 offsets at a time, and with the first 32 of them
// the row's own number (a request a row). off[0] <= t < off[B] or -1; ends for any contents of off.
__device__ __forceinline__ int32_t request_by_warp(const uint32_t* off, uint32_t B, uint32_t t) {
    if (!off) return (int32_t)t;
    const uint32_t lane = threadIdx.x & 31, guess = min(t, B - 1);
    uint32_t lo = 0, n = B, step = (n + 31) / 32;  // off[lo] <= t < off[lo + n]
    const uint32_t probe = off[lane == 0 ? guess : lane == 1 ? guess + 1 : lane == 2 ? 0 : B];
    uint32_t first = off[min(lane * step, B)];
    const uint32_t at = __shfl_sync(0xFFFFFFFFu, probe, 0), after = __shfl_sync(0xFFFFFFFFu, probe, 1);
    if (at <= t && t < after) return (int32_t)guess;
    if (__shfl_sync(0xFFFFFFFFu, probe, 2) > t || __shfl_sync(0xFFFFFFFFu, probe, 3) <= t) return -1;
    while (n > 1) {
        const uint32_t below = __ballot_sync(0xFFFFFFFFu, lane * step < n && first <= t);
        const uint32_t k = 31 - __clz(below | 1u);  // the last probe that is not past t
        lo += k * step;
        n = min(step, n - k * step);
        step = (n + 31) / 32;
        if (n > 1) first = off[lo + (lane * step < n ? lane * step : 0)];
    }
    return (int32_t)lo;
}

// One warp describes row t; loads that do not need each other's values are started together.
__device__ __forceinline__ void describe(const ProcessParams& p, uint32_t t, Row* row, bool mask_fits, bool report) {
    const uint32_t lane = threadIdx.x & 31;
    const int32_t b = request_by_warp(p.row_offsets, p.B, t);
    if (lane != 0) return;
    Row r = {b, 0u, 0u, 0u, 0u, 0u, 0u, {1.f, 1.f, 0.f, 0.f}};
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
        if (!mask_fits) r.request = -1;
        if (r.prompt > r.h1 - r.h0) r.prompt = r.h1 - r.h0;
    }
    if (r.request < 0 && report) flag(p.status, code);
    *row = r;
}

// A stretch of tokens that a CTA looks at: the request's history, or what a sorted chunk of it
// has in the slice.
struct Tokens {
    const uint32_t* at;
    uint32_t n;
    uint32_t prompt;  // history: its first tokens are the prompt; sorted: bit 31 tells
    bool sorted;
    __device__ __forceinline__ uint32_t token(uint32_t entry) const { return sorted ? entry & 0x7FFFFFFFu : entry; }
    __device__ __forceinline__ bool in_prompt(uint32_t i, uint32_t entry) const {
        return sorted ? entry >> 31 : i < prompt;
    }
};

// The table of tokens [lo, lo + size): a word of 16 bits (WIDE: 32) a token.
template <bool WIDE>
struct Table {
    uint32_t* words;
    uint32_t lo, size;
    static constexpr uint32_t kAll = WIDE ? 0xFFFFFFFFu : 0xFFFFu;
    static constexpr uint32_t kPrompt = WIDE ? 0x80000000u : 0x8000u;
    __device__ __forceinline__ uint32_t shift(uint32_t slot) const { return WIDE ? 0 : slot % 2 * 16; }
    __device__ __forceinline__ uint32_t* word(uint32_t slot) const { return words + (WIDE ? slot : slot / 2); }

    __device__ __forceinline__ uint32_t count(const Tokens& s, uint32_t i, uint32_t entry) const {  // 1: of the slice
        const uint32_t slot = s.token(entry) - lo;
        if (slot >= size) return 0;
        if (s.in_prompt(i, entry)) atomicOr(word(slot), kPrompt << shift(slot));
        else atomicAdd(word(slot), 1u << shift(slot));
        return 1;
    }
    // The token's word, for the first thread that asks (0 for others), which empties it.
    __device__ __forceinline__ uint32_t take(uint32_t slot) const {
        if (slot >= size) return 0;
        if (!(*static_cast<volatile uint32_t*>(word(slot)) >> shift(slot) & kAll)) return 0;
        return atomicAnd(word(slot), ~(kAll << shift(slot))) >> shift(slot) & kAll;
    }
};

// Ask for a row's slice in L2, thread `k` of `threads`.
template <typename T>
__device__ __forceinline__ void prefetch_slice(const T* row, uint32_t lo, uint32_t hi, uint32_t k, uint32_t threads) {
    constexpr uint32_t kPiece = 4096;
    const uintptr_t from = (reinterpret_cast<uintptr_t>(row + lo) + 15) & ~(uintptr_t)15;
    const uintptr_t to = reinterpret_cast<uintptr_t>(row + hi) & ~(uintptr_t)15;
    for (uintptr_t at = from + k * kPiece; at < to; at += threads * kPiece) {
        const uint32_t bytes = to - at < kPiece ? (uint32_t)(to - at) : kPiece;
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
    }
}

constexpr uint32_t kSortThreads = 512;
constexpr uint32_t kSortEach = kChunk / kSortThreads;
constexpr uint32_t kNowhere = 0xFFFF0000u;

// Histories are sorted in chunks of kChunk tokens. Request b's chunk c has number
// b + h0 / kChunk + c: no two have the same, and there are at most B + total / kChunk + 1, as long
// as the offsets nowhere decrease. Where they do, two requests may claim one number, or a part of
// `sorted` each, and a chunk may have no CTA that finds it (its bounds would be an earlier call's).
// So one CTA looks at all offsets and writes the verdict into a word of the workspace, and where
// they are bad every row reads its history as it is, as without the sort.
__device__ __forceinline__ uint32_t first_chunk(const ProcessParams& p, uint32_t b) {
    return b + p.history_offsets[b] / kChunk;
}

// Sort a chunk by slices: sorted[h0 + c kChunk ...] gets its tokens (bit 31: of the prompt),
// bounds[chunk][k] where slice k's begin. A warp takes the places of its tokens of one slice
// together; their order within a slice is left open. grid: a CTA a chunk, and one for the verdict
__global__ void __launch_bounds__(kSortThreads, 3) k_sort_history(ProcessParams p) {
    __shared__ uint32_t place[kMaxSlices + 1];
    __shared__ uint32_t s_request;
    pdl_wait();
    pdl_trigger();  // after the wait: the copy may read logits, which are complete now
    const uint32_t tid = threadIdx.x, lane = tid & 31, chunk = blockIdx.x;
    if (chunk == gridDim.x - 1) {
        bool falls = false;
        for (uint32_t b = tid; b < p.B; b += kSortThreads) falls |= p.history_offsets[b] > p.history_offsets[b + 1];
        falls = __syncthreads_or(falls);
        if (tid == 0) p.status[kOrderedWord] = !falls;
        return;
    }
    for (uint32_t k = tid; k <= p.slices; k += kSortThreads) place[k] = 0;
    if (tid < 32) {  // the last request whose first chunk is not past this one, 32 at a time
        uint32_t lo = 0, n = p.B;
        while (n > 1) {
            const uint32_t step = (n + 31) / 32, i = lane * step;
            const uint32_t below = __ballot_sync(0xFFFFFFFFu, i < n && first_chunk(p, lo + (i < n ? i : 0)) <= chunk);
            const uint32_t k = 31 - __clz(below | 1u);
            lo += k * step;
            n = min(step, n - k * step);
        }
        if (lane == 0) s_request = lo;
    }
    __syncthreads();
    const uint32_t b = s_request, h0 = p.history_offsets[b], h1 = p.history_offsets[b + 1];
    const bool neutral = (!p.repetition || p.repetition[b] == 1.f) && (!p.frequency || p.frequency[b] == 0.f) &&
                         (!p.presence || p.presence[b] == 0.f);
    const uint32_t before = chunk - first_chunk(p, b);  // chunks of the request before this one
    if (neutral || h0 > h1 || h1 > p.history_total || chunk < first_chunk(p, b) ||
        (uint64_t)before * kChunk >= h1 - h0)
        return;  // (no chunk, or not read: see describe)
    const uint32_t from = before * kChunk, n = min(kChunk, h1 - h0 - from);
    const uint32_t prompt = p.prompt_lens ? p.prompt_lens[b] : 0u;
    uint32_t v[kSortEach], where[kSortEach];  // where: slice << 16 | place among the chunk's of the slice
    bool outside = false;
#pragma unroll
    for (uint32_t k = 0; k < kSortEach; ++k) {
        const uint32_t i = tid + k * kSortThreads;
        v[k] = i < n ? p.history[h0 + from + i] : 0u;
    }
#pragma unroll
    for (uint32_t k = 0; k < kSortEach; ++k) {
        const uint32_t i = tid + k * kSortThreads;
        const uint32_t slice = i < n && v[k] < p.V ? v[k] / p.slice : kNowhere >> 16;
        outside |= i < n && v[k] >= p.V;
        if (from + i < prompt) v[k] |= 0x80000000u;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, slice), rank = __popc(peers & ((1u << lane) - 1u));
        uint32_t at = 0;
        if (slice != kNowhere >> 16 && rank == 0) at = atomicAdd(place + slice + 1, __popc(peers));
        where[k] = slice << 16 | (__shfl_sync(0xFFFFFFFFu, at, __ffs(peers) - 1) + rank);
    }
    __syncthreads();
    if (tid < 32) {  // place[k]: tokens of the slices before k
        uint32_t sum = 0;
        for (uint32_t k0 = 0; k0 <= p.slices; k0 += 32) {
            uint32_t x = k0 + lane <= p.slices ? place[k0 + lane] : 0u;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
                if (lane >= d) x += y;
            }
            x += sum;
            if (k0 + lane <= p.slices) {
                place[k0 + lane] = x;
                p.bounds[(uint64_t)chunk * (p.slices + 1) + k0 + lane] = x;
            }
            sum = __shfl_sync(0xFFFFFFFFu, x, 31);
        }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t k = 0; k < kSortEach; ++k)
        if (where[k] < kNowhere) p.sorted[h0 + from + place[where[k] >> 16] + (where[k] & 0xFFFF)] = v[k];
    if (outside) flag(p.status, LP_ERR_TOKEN_RANGE);
}

// Offsets of n lists within `total`, by a whole CTA: LP_ERR_OFFSETS where they decrease or pass it.
__device__ __forceinline__ void check_offsets(const uint32_t* off, uint32_t n, uint32_t total, uint32_t* status) {
    bool bad = threadIdx.x == 0 && off[n] > total;
    for (uint32_t i = threadIdx.x; i < n; i += blockDim.x) bad |= off[i] > off[i + 1];
    if (bad) flag(status, LP_ERR_OFFSETS);
}

// Threads of a CTA. With sorted histories more, which overlap better (256 x 128256 f32, histories
// of 30000: 256 threads 69.0 us, 384 66.1); without, the registers they leave cost more (240 x
// 152064 bf16, histories of 1000: 47.1 and 51.2 us).
__host__ __device__ constexpr uint32_t threads(bool sorted) { return sorted ? 384 : 256; }

// grid: T x slices CTAs, and one more that looks at the lists' offsets as a whole (a row's CTAs only
// see its own request's). All rows' first slices first: a vocabulary's frequent tokens mostly have
// its low numbers, and the CTAs with the most to count should not be the last to start (256 rows
// with histories of 30000: 80 us row by row, 69 so).
// Without sorted histories at most 48 registers, so that five CTAs share an SM where the slices are
// short enough (240 x 152064 bf16: 52.8 us with 55 registers, 45.3 so).
template <typename T, bool VEC, bool SORTED>
__global__ void __launch_bounds__(threads(SORTED), SORTED ? kResident : kResident + 1) k_process(ProcessParams p) {
    constexpr uint32_t kThreads = threads(SORTED);
    extern __shared__ __align__(16) uint32_t table[];  // slice / 2 words
    __shared__ Row s_row;
    __shared__ uint32_t s_in_slice;
    __shared__ uint32_t s_mask[kMaxSlice / 32 + 2];    // mask words of the slice
    pdl_trigger();
    const uint32_t tid = threadIdx.x;
    const uint32_t part = blockIdx.x / p.T, t = blockIdx.x - part * p.T;
    if (part == p.slices) {
        if constexpr (!SORTED) pdl_wait();
        if (p.row_offsets) check_offsets(p.row_offsets, p.B, p.T, p.status);
        if (p.history) check_offsets(p.history_offsets, p.B, p.history_total, p.status);
        if (p.bias_tokens) check_offsets(p.bias_offsets, p.B, p.bias_total, p.status);
        return;
    }
    const uint32_t lo = part * p.slice, hi = min(lo + p.slice, p.V);  // this CTA's tokens
    const T* in = static_cast<const T*>(p.logits) + (uint64_t)t * p.stride;
    float* out = p.out + (uint64_t)t * p.out_stride;
    const float ninf = __int_as_float(0xff800000);
    if (p.history)
        for (uint32_t i = tid; i < (p.slice + 7) / 8; i += kThreads) reinterpret_cast<uint4*>(table)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) s_in_slice = 0;
    if constexpr (!SORTED) pdl_wait();  // (the sort has waited for what logits and the lists come from)
    // One warp finds out whose the row is; the others, at the same time, whether it is masked, and
    // read its mask or ask for the slice.
    const int64_t m = !p.mask ? -1 : p.mask_index ? (int64_t)p.mask_index[t] : (int64_t)t;
    const bool mask_fits = m < (int64_t)p.mask_rows, masked = m >= 0 && mask_fits;
    const uint32_t word0 = lo >> 5, words = ((hi - 1) >> 5) - word0 + 1;
    if (tid < 32) {
        describe(p, t, &s_row, mask_fits, part == 0);
    } else if (masked) {
        const uint32_t* mask = p.mask + m * (int64_t)p.mask_stride + word0;
        for (uint32_t i = tid - 32; i <= words; i += kThreads - 32)  // (the last is read beside the one before)
            s_mask[i] = i < words ? mask[i] : 0u;
    } else {
        prefetch_slice(in, lo, hi, tid - 32, kThreads - 32);
    }
    __syncthreads();
    const Row row = s_row;
    if constexpr (SORTED) pdl_wait();
    const bool ordered = !SORTED || __ldcg(p.status + kOrderedWord) != 0;
    if (row.request < 0) {
        for (uint32_t v = lo + tid; v < hi; v += kThreads) out[v] = __int_as_float(0x7fffffff);
        return;
    }
    const auto allowed = [&](uint32_t v) { return !masked || ((s_mask[(v >> 5) - word0] >> (v & 31)) & 1u); };
    // 15 bits hold any count of an output part of up to 32767 tokens
    const bool wide = row.counted && row.h1 - row.h0 - row.prompt > 0x7FFFu;
    const Table<false> counts = {table, lo, hi - lo};
    const uint32_t pieces = !row.counted ? 0 : SORTED ? (row.h1 - row.h0 + kChunk - 1) / kChunk : 1;
    const auto piece = [&](uint32_t c) -> Tokens {
        if (!SORTED) return {p.history + row.h0, row.h1 - row.h0, row.prompt, false};
        if (!ordered) {  // (in the same pieces)
            const uint32_t from = c * kChunk;
            return {p.history + row.h0 + from, min(kChunk, row.h1 - row.h0 - from), row.prompt - min(row.prompt, from), false};
        }
        const uint32_t* bounds = p.bounds + (uint64_t)(row.request + row.h0 / kChunk + c) * (p.slices + 1) + part;
        const uint32_t limit = min(kChunk, row.h1 - row.h0 - c * kChunk);
        const uint32_t from = min(bounds[0], limit), to = min(bounds[1], limit);
        return {p.sorted + row.h0 + (uint64_t)c * kChunk + from, to > from ? to - from : 0u, 0u, true};
    };
    // Sorted pieces side by side, a warp each with 8 tokens a lane in flight, since a piece's loads
    // wait for each other (256 histories of 30000: 72 us; one after the other by all threads, 4 in
    // flight: 80). A history that is not sorted is one piece, and short: 8 in flight cost it 7 %.
    constexpr uint32_t kTeam = SORTED ? 32 : kThreads, kTeams = kThreads / kTeam, kHeld = SORTED ? 8 : 4;
    const uint32_t my_team = SORTED ? tid >> 5 : 0, me = SORTED ? tid & 31 : tid;
    bool outside = false;
    uint32_t mine = 0;  // tokens of the slice that this thread has counted
    const auto count_all = [&](const auto& into) {
        for (uint32_t c = my_team; c < pieces; c += kTeams) {
            const Tokens s = piece(c);
            for (uint32_t i0 = me; i0 < s.n; i0 += kHeld * kTeam) {
                uint32_t e[kHeld];
#pragma unroll
                for (uint32_t k = 0; k < kHeld; ++k) e[k] = i0 + k * kTeam < s.n ? s.at[i0 + k * kTeam] : 0u;
#pragma unroll
                for (uint32_t k = 0; k < kHeld; ++k) {
                    if (i0 + k * kTeam >= s.n) break;
                    outside |= s.token(e[k]) >= p.V;
                    mine += into.count(s, i0 + k * kTeam, e[k]);
                }
            }
        }
    };
    // Many tokens of the slice in the table (1 in 32): looked at during the copy. (256 rows of
    // 128256 with histories of 30000: 1 in 32 71.9 us, 1 in 16 73.2, 1 in 12 73.8.)
    bool dense = false;
    if (row.counted && !wide) {
        count_all(counts);
        mine = __reduce_add_sync(0xFFFFFFFFu, mine);
        if (tid % 32 == 0 && mine) atomicAdd(&s_in_slice, mine);
        __syncthreads();
        dense = s_in_slice > (hi - lo) / 32;
    }
    // this thread's first bias, long before it is needed
    const bool biased = row.b1 - row.b0 > tid;
    const uint32_t bias_at = biased ? p.bias_tokens[row.b0 + tid] : 0u;
    const float bias = biased ? p.bias_values[row.b0 + tid] : 0.f;

    // the copy
    const uint32_t first = VEC ? min(lo + ((-(uint32_t)(reinterpret_cast<uintptr_t>(out + lo) >> 2)) & 3u), hi) : hi;
    const uint32_t vecs = (hi - first) / 4, vec_end = first + 4 * vecs;
    const auto one = [&](uint32_t v) {
        const uint32_t w = dense ? *counts.word(v - lo) >> counts.shift(v - lo) & 0xFFFFu : 0u;
        out[v] = !allowed(v) ? ninf : w ? penalised(to_f32(in[v]), w & 0x7FFF, row.q) : to_f32(in[v]);
    };
    for (uint32_t v = lo + tid; v < first; v += kThreads) one(v);
    for (uint32_t v = vec_end + tid; v < hi; v += kThreads) one(v);
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
                if (dense) {
                    // the words of 4 tokens from slot 4 i + (first - lo) on: out of two or three
                    const uint32_t slot = first - lo + 4 * i, odd = slot % 2 * 16;
                    const uint32_t* w = table + slot / 2;
                    const uint32_t w0 = __funnelshift_r(w[0], w[1], odd), w1 = __funnelshift_r(w[1], w[odd ? 2 : 1], odd);
                    if (w0 & 0xFFFF) y.x = penalised(y.x, w0 & 0x7FFF, row.q);
                    if (w0 >> 16) y.y = penalised(y.y, w0 >> 16 & 0x7FFF, row.q);
                    if (w1 & 0xFFFF) y.z = penalised(y.z, w1 & 0x7FFF, row.q);
                    if (w1 >> 16) y.w = penalised(y.w, w1 >> 16 & 0x7FFF, row.q);
                }
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

    // few tokens of the history: corrected now
    const auto correct = [&](const auto& from) {
        for (uint32_t c = my_team; c < pieces; c += kTeams) {
            const Tokens s = piece(c);
            for (uint32_t i0 = me; i0 < s.n; i0 += kHeld * kTeam) {
                uint32_t v[kHeld], w[kHeld];
                float x[kHeld];
#pragma unroll
                for (uint32_t k = 0; k < kHeld; ++k) v[k] = i0 + k * kTeam < s.n ? s.token(s.at[i0 + k * kTeam]) : p.V;
#pragma unroll
                for (uint32_t k = 0; k < kHeld; ++k) {
                    w[k] = v[k] < p.V ? from.take(v[k] - from.lo) : 0u;
                    if (w[k] && !allowed(v[k])) w[k] = 0;
                }
#pragma unroll
                for (uint32_t k = 0; k < kHeld; ++k) x[k] = w[k] ? out[v[k]] : 0.f;
#pragma unroll
                for (uint32_t k = 0; k < kHeld; ++k)
                    if (w[k]) out[v[k]] = penalised(x[k], w[k] & (from.kPrompt - 1), row.q);
            }
        }
    };
    if (row.counted && !wide && !dense) {
        __syncthreads();
        correct(counts);
    } else if (wide) {
        const uint32_t half = (p.slice + 7) / 8 * 4;  // (a table of 16 bits a token holds half as many of 32)
        for (uint32_t first_token = lo; first_token < hi; first_token += half) {
            const Table<true> wide_counts = {table, first_token, min(half, hi - first_token)};
            count_all(wide_counts);
            __syncthreads();
            correct(wide_counts);
            __syncthreads();
        }
    }
    if (outside && part == 0) flag(p.status, LP_ERR_TOKEN_RANGE);
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
std::atomic<uint64_t> g_smem_set[2][2];

template <typename T>
lp_status launch_process(const ProcessParams& p, bool vec, unsigned ctas, lp_stream_t s) {
    const bool sorted = p.sorted != nullptr;
    void (*kernel)(ProcessParams) = sorted ? vec ? k_process<T, true, true> : k_process<T, false, true>
                                           : vec ? k_process<T, true, false> : k_process<T, false, false>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), kMaxSlice * 2 + 16, &g_smem_set<T>[vec][sorted])) return LP_ERR_CUDA;
    return launch(kernel, dim3(ctas), threads(sorted), (size_t)p.slice * 2 + 16, s, 1, p);
}

}  // namespace

extern "C" size_t lp_head_process_workspace_size(uint32_t B, uint32_t history_total) {
    // Of the calls of up to so many requests and tokens the one that needs most: histories are sorted
    // where their mean is kSortFrom, so the requests that count are at most total / kSortFrom.
    const size_t requests = history_total / kSortFrom < B ? history_total / kSortFrom : B;
    if (requests == 0) return kHeaderBytes;
    return kHeaderBytes + ((requests + history_total / kChunk + 1) * (kMaxSlices + 1) + history_total) * 4;
}

extern "C" lp_status lp_head_process(const void* logits, uint32_t dtype, uint32_t T, uint32_t V, uint64_t stride,
                                     const uint32_t* row_offsets, uint32_t B, const uint32_t* history,
                                     const uint32_t* history_offsets, uint32_t history_total,
                                     const uint32_t* prompt_lens, const float* repetition, const float* frequency,
                                     const float* presence, const uint32_t* bias_tokens, const float* bias_values,
                                     const uint32_t* bias_offsets, uint32_t bias_total, const uint32_t* mask,
                                     uint64_t mask_stride, uint32_t mask_rows, const int32_t* mask_index, float* out,
                                     uint64_t out_stride, void* workspace, size_t workspace_bytes,
                                     lp_stream_t stream) {
    if (T == 0 || V == 0 || B == 0) return LP_ERR_SHAPE;  // (before the pointers: an empty tensor has none)
    if (!logits || !out || (history && !history_offsets) ||
        (bias_tokens && (!bias_values || !bias_offsets)))
        return LP_ERR_NULL;
    if (!workspace || workspace_bytes < kHeaderBytes || !aligned_to(workspace, 256)) return LP_ERR_WORKSPACE;
    if (dtype > LP_F16) return LP_ERR_DTYPE;
    if (V >= 0x7FFFFFFFu || stride < V || out_stride < V)
        return LP_ERR_SHAPE;
    if (!row_offsets && B != T) return LP_ERR_SHAPE;
    if (mask && (mask_rows == 0 || mask_rows > 0x7FFFFFFFu || mask_stride < ((uint64_t)V + 31) / 32 ||
                 (!mask_index && mask_rows < T)))
        return LP_ERR_SHAPE;
    const size_t e = dtype_bytes(dtype);
    if (!aligned_to(logits, e)) return LP_ERR_SHAPE;
    for (const void* ptr : {static_cast<const void*>(out), static_cast<const void*>(row_offsets),
                            static_cast<const void*>(history), static_cast<const void*>(history_offsets),
                            static_cast<const void*>(prompt_lens), static_cast<const void*>(repetition),
                            static_cast<const void*>(frequency), static_cast<const void*>(presence),
                            static_cast<const void*>(bias_tokens), static_cast<const void*>(bias_values),
                            static_cast<const void*>(bias_offsets), static_cast<const void*>(mask),
                            static_cast<const void*>(mask_index)})
        if (!aligned_to(ptr, 4)) return LP_ERR_SHAPE;
    if (static_cast<const void*>(out) == logits && (dtype != LP_F32 || stride != out_stride)) return LP_ERR_SHAPE;
    const int sms = sm_count();
    if (sms == 0) return LP_ERR_CUDA;
    ProcessParams p = {};
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
        if (slices > kMaxSlices) slices = kMaxSlices;
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
    const uint64_t ctas = (uint64_t)p.slices * T + (row_offsets || p.history || p.bias_tokens);
    if (ctas > 0x7FFFFFFFull) return LP_ERR_SHAPE;
    // Long histories are sorted by slices first; below that, reading them in every CTA costs less
    // than a second kernel. Rows of 128256 f32, all histories of one length, us (sorted | not):
    //     256 rows  2000: 60 | 59    4000: 64 | 70    8000: 72 | 89   16000: 78 | 113
    //      32 rows  2000: 21 | 17    4000: 27 | 21    8000: 27 | 27   16000: 29 | 36
    //       4 rows  2000: 17 | 13    4000: 21 | 15    8000: 21 | 17   16000: 21 | 25
    if (p.history && history_total / B >= kSortFrom && p.slices <= kMaxSlices) {
        if (workspace_bytes < lp_head_process_workspace_size(B, history_total)) return LP_ERR_WORKSPACE;
        p.bounds = reinterpret_cast<uint32_t*>(static_cast<unsigned char*>(workspace) + kHeaderBytes);
        const uint32_t chunks = B + history_total / kChunk + 1;
        p.sorted = p.bounds + (size_t)chunks * (p.slices + 1);
        const lp_status st = launch(k_sort_history, dim3(chunks + 1), kSortThreads, 0, stream, 1, p);
        if (st != LP_OK) return st;
    }
    // 4 values at a time where logits and out have their 4-value boundaries at the same tokens
    const bool vec = stride % 4 == out_stride % 4 &&
                     (reinterpret_cast<uintptr_t>(logits) / e) % 4 == (reinterpret_cast<uintptr_t>(out) / 4) % 4;
    if (dtype == LP_F32) return launch_process<float>(p, vec, (unsigned)ctas, stream);
    if (dtype == LP_BF16) return launch_process<__nv_bfloat16>(p, vec, (unsigned)ctas, stream);
    return launch_process<__half>(p, vec, (unsigned)ctas, stream);
}
