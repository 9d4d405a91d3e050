// First kernel of the projection with adapters: u[t, j] = s_a sx[t] sum_h x[t, h] A_a[j, h],
// and for each tile of rows the list of its adapters (lp_adapters.h).
//
// Two forms. A block a row, its warps taking the row's dot products in turn: each reads the
// rows of its adapter's A, so it suits rows with adapters of their own (decode). A block of 16
// rows, which multiplies them by the A of every adapter among them on the tensor cores
// (mma.sync: the work is too small and too ragged for a pipeline of its own): long requests,
// where 16 rows have one adapter or two (launch_shrink has both sides' times). Bound by latency:
// 2048 rows of 8 requests, rank 64, H = 4096 take 30 us, of which x and A at HBM's rate would be
// 3; the product runs meanwhile and asks for u at the end of its first tile.
#include "lp_adapters.h"

namespace {

using namespace lph;

constexpr uint32_t kThreads = 512;
constexpr uint32_t kWarps = kThreads / 32;
constexpr uint32_t kBlockRows = 16;

__device__ __forceinline__ void load_x8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(w[i], __nv_bfloat16());
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load_x8(const __half* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(w[i], __half());
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load_x8(const __nv_fp8_e4m3* p, float (&v)[8]) {
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    const uint32_t w[2] = {a.x, a.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((uint16_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}


// The adapter of row t (negative: none); a bad id or a row of no request: adapter 0 and *bad.
__device__ __forceinline__ int32_t adapter_of(const ShrinkParams& p, uint32_t t, bool* bad, uint32_t* code) {
    const int b = request_of(p.row_offsets, p.B, t);
    const int32_t a = b < 0 ? 0 : p.adapter_ids[b];
    *bad = b < 0 || a >= (int32_t)p.adapters;
    *code = b < 0 ? LP_ERR_OFFSETS : LP_ERR_ADAPTER;
    return *bad ? 0 : max(a, -1);
}

// The lists of one tile of rows; a thread a row (the block's first kMaxTileT).
__device__ void list_tile(const ShrinkParams& p, uint32_t tile) {
    __shared__ int32_t id[kMaxTileT];
    __shared__ uint32_t key[kMaxTileT];       // of a listed row: the first listed row with its adapter
    __shared__ uint8_t begins_at[kMaxTileT];  // by place: an item begins here
    constexpr uint32_t kUnlisted = kMaxTileT + 1;
    if (threadIdx.x >= kMaxTileT) return;
    const auto sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kMaxTileT) : "memory"); };
    const uint32_t c = threadIdx.x, t0 = tile * p.tile_t, rows = min(p.tile_t, p.T - t0);
    bool bad;
    uint32_t code;
    id[c] = c < rows ? adapter_of(p, t0 + c, &bad, &code) : -2;
    sync();
    TileGroups* g = reinterpret_cast<TileGroups*>(p.groups + (size_t)tile * kGroupBytes);
    // the warp's rows are one block: its first adapter, its second, and whether there are more
    constexpr uint32_t kAll = 0xFFFFFFFFu;
    const int32_t mine = id[c];
    const uint32_t with = __ballot_sync(kAll, mine >= 0), in = __ballot_sync(kAll, c < rows);
    const int32_t a0 = __shfl_sync(kAll, mine, with ? __ffs(with) - 1 : 0);
    const uint32_t m0 = with ? __ballot_sync(kAll, mine == a0) : 0u, rest = with & ~m0;
    const int32_t a1 = __shfl_sync(kAll, mine, rest ? __ffs(rest) - 1 : 0);
    const uint32_t m1 = rest ? __ballot_sync(kAll, mine == a1) : 0u;
    const bool many = with && (!p.tensor || (rest & ~m1) != 0);
    __shared__ uint32_t adapter[3][kBlocks], listed_bits;  // of pass 0, of pass 1: first and second
    if (c == 0) listed_bits = 0;
    sync();
    if (c % kBlock == 0) {
        const uint32_t b = c / kBlock, pass = m0 == in && !p.apart ? 0 : 1;  // of the first adapter
        const bool tensor = with && !many;
        adapter[0][b] = tensor && pass == 0 ? (uint32_t)a0 : kNoAdapter;
        adapter[1][b] = tensor && pass == 1 ? (uint32_t)a0 : kNoAdapter;
        adapter[2][b] = tensor && rest ? (uint32_t)a1 : kNoAdapter;
        g->rows[0][b] = m0;
        g->rows[1][b] = m1;
        if (many) atomicOr(&listed_bits, 1u << b);
    }
    sync();
    if (c == 0) {
        uint32_t runs = 0, blocks = 0, second = 0, place = 0, taken = 0;
        for (uint32_t b = 0; b < kBlocks; ++b)
            if (adapter[1][b] != kNoAdapter) taken |= 1u << b;
        for (uint32_t b = 0; b < kBlocks; ++b) {
            if (adapter[2][b] == kNoAdapter) continue;
            const uint32_t free = ~taken & ((1u << p.tile_t / kBlock) - 1u);
            if (free) {
                const uint32_t f = __ffs(free) - 1;
                taken |= 1u << f;
                place |= f << 4 * b;
                second |= 1u << b;
            } else {
                adapter[1][b] = adapter[2][b] = kNoAdapter;
                listed_bits |= 1u << b;
            }
        }
        for (uint32_t pass = 0; pass < 2; ++pass) {
            for (uint32_t b0 = 0, n; b0 < kBlocks; b0 += n) {
                const uint32_t a = adapter[pass][b0];
                for (n = 1; b0 + n < kBlocks && adapter[pass][b0 + n] == a; ++n) {}
                if (a == kNoAdapter) continue;
                g->run[runs++] = make_uint2(b0 << 24 | pass << 16 | b0 << 8 | n, a);
                if (pass) blocks |= ((1u << n) - 1u) << b0;
            }
        }
        for (uint32_t b = 0; b < kBlocks; ++b)
            if (second >> b & 1) g->run[runs++] = make_uint2((place >> 4 * b & 15) << 24 | 1u << 16 | b << 8 | 1u, adapter[2][b]);
        g->blocks = blocks;
        g->second = second;
        g->place = place;
        g->runs = runs;
        g->listed = listed_bits;
    }
    sync();
    const bool listed = listed_bits >> (c / kBlock) & 1;
    uint32_t k = kUnlisted;
    key[c] = listed && c < rows ? 0 : kUnlisted;
    sync();
    if (key[c] != kUnlisted) {
        k = kMaxTileT;  // rows without an adapter come last
        if (id[c] >= 0)
            for (k = 0; id[k] != id[c] || key[k] == kUnlisted; ++k) {}
    }
    sync();
    key[c] = k;
    begins_at[c] = 0;
    sync();
    // place of this row in the order by (key, own place)
    uint32_t place = 0, among = 0, total = 0;
    for (uint32_t i = 0; i < rows; ++i) {
        const bool same_before = key[i] == k && i < c;
        place += key[i] < k || same_before;
        among += same_before;
        total += key[i] != kUnlisted;
    }
    const bool begins = k != kUnlisted && among % kItemRows == 0;
    if (begins) begins_at[place] = 1;
    sync();
    if (k != kUnlisted) g->order[place] = (uint8_t)c;
    if (begins) {
        uint32_t item = 0, size = 1;
        for (uint32_t i = 0; i < place; ++i) item += begins_at[i];
        while (place + size < total && !begins_at[place + size]) ++size;
        g->item[item] = id[c] < 0 ? kNoAdapter : (uint32_t)id[c];
        g->start[item] = (uint8_t)place;
        g->size[item] = (uint8_t)size;
        if (place + size == total) g->items = item + 1;
    }
    if (c == 0 && total == 0) g->items = 0;
}

// The part-th of the three 16-bit values whose sum is v: rounded towards zero, so that all have v's
// sign, and none is zero while v is not: a value that rounds to itself leaves its last place to the
// next part. An infinite element of B then gives u B's infinity (a part of zero would give 0 x inf =
// NaN), and so does an infinite u. bf16 parts hold v's 24 bits. f16 parts hold it to 2^-24 at least,
// v's largest in the row being 2^13 or more: elements below 2^-38 of the row's largest are lost, and
// below 2^-35 the parts can be zero.
__device__ __forceinline__ uint16_t part_of(float v, uint32_t part, bool f16) {
    const uint32_t sign = __float_as_uint(v) >> 16 & 0x8000u;
    float m = fabsf(v);
    if (!(m < __int_as_float(0x7f800000)))
        return f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
    if (f16 && m < 1.f) m = rintf(m * 16777216.f) * 5.9604644775390625e-8f;  // whole multiples of 2^-24
    for (uint32_t n = 0;; ++n) {
        uint32_t h = f16 ? __half_as_ushort(__float2half_rz(m)) : __float_as_uint(m) >> 16;
        const auto value = [&] { return f16 ? __half2float(__ushort_as_half((uint16_t)h)) : __uint_as_float(h << 16); };
        // what the others need: the second and third f16 part 2^-24 each
        if (n < 2 && m - value() < (f16 && n == 0 ? 1.1920928955078125e-7f : 1.0e-45f)) {
            const uint32_t step = f16 && n == 0 && h <= 0x0800u ? 2 : 1;  // (places of 2^-24 up to there)
            if (h > step) h -= step;
        }
        if (n == part) return (uint16_t)(h | sign);
        m -= value();
    }
}

// One warp writes row t's u (u[0, rank) in shared memory, zero past the rank), and its parts.
__device__ void write_row(const ShrinkParams& p, uint32_t t, const float* u) {
    const uint32_t lane = threadIdx.x & 31, cols = rank_cols(p.rank);
    float top = 0.f;
    for (uint32_t j = lane; j < cols; j += 32) {
        p.u[(uint64_t)t * cols + j] = u[j];
        if (fabsf(u[j]) < __int_as_float(0x7f800000)) top = fmaxf(top, fabsf(u[j]));
    }
    if (!p.tensor) return;
    // f16 parts: u as values times a power of two, the row's largest (that is finite) in [2^13,
    // 2^14), so that neither their size nor the third part leaves f16's range. bf16 has f32's.
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const int e = p.lora_f16 && top > 0.f ? ilogbf(top) - 13 : 0;
    if (lane == 0) p.factor[t] = ldexpf(1.f, e);
    const uint32_t width = part_cols(p.rank);
    if (lane >= part_rows(p.rank) * 8) return;
    const uint32_t line = lane / 8, first = line * 64 + lane % 8 * 8;  // a piece of 8 columns
    const uint32_t part = first / width, j0 = first - part * width;
    uint16_t piece[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        piece[q] = part > 2 || j0 + q >= p.rank ? 0 : part_of(ldexpf(u[j0 + q], -e), part, p.lora_f16);
    }
    *reinterpret_cast<uint4*>(p.parts + ((uint64_t)line * p.part_stride + t) * 64 + lane % 8 * 8) =
        make_uint4(piece[0] | (uint32_t)piece[1] << 16, piece[2] | (uint32_t)piece[3] << 16,
                   piece[4] | (uint32_t)piece[5] << 16, piece[6] | (uint32_t)piece[7] << 16);
}

__device__ __forceinline__ float row_scale(const ShrinkParams& p, uint32_t t, int32_t a) {
    const float s = p.adapter_scale ? p.adapter_scale[a] : 1.f;
    return p.x_scale ? s * p.x_scale[t] : s;
}

// Ask for a row in L2 (its start and bytes are multiples of 16), piece `k` of 1 KB and every
// `step`-th after it: the loads that follow wait for HBM once, not once a round (48 rows, H =
// 4096, rank 32: 13 -> 10 us, and the whole projection of 152064 e4m3 136 -> 127 us; for blocks of
// 16 rows it gained nothing).
__device__ __forceinline__ void prefetch_row(const void* row, uint32_t bytes, uint32_t k, uint32_t step) {
    for (uint32_t at = k * 1024; at < bytes; at += step * 1024)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const unsigned char*>(row) + at),
                     "r"(min(1024u, bytes - at))
                     : "memory");
}

// grid: T blocks, one a row, then one a tile for its lists.
template <typename X, typename A>
__global__ void __launch_bounds__(1024) k_shrink_row(ShrinkParams p) {
    __shared__ float s_u[64];
    pdl_wait();
    pdl_trigger();  // after the wait: the product kernel may read x, which is complete now
    if (blockIdx.x >= p.T) {
        list_tile(p, blockIdx.x - p.T);
        return;
    }
    const uint32_t warps = blockDim.x >> 5;
    const uint32_t t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const X* x = static_cast<const X*>(p.x) + (uint64_t)t * p.x_stride;
    if (warp == 0) prefetch_row(x, p.H * sizeof(X), lane, 32);
    bool bad;
    uint32_t code;
    const int32_t a = adapter_of(p, t, &bad, &code);
    if (bad && threadIdx.x == 0) flag(p.status, code);
    const uint32_t cols = rank_cols(p.rank);
    if (a >= 0)
        for (uint32_t j = warp; j < p.rank; j += warps)
            prefetch_row(static_cast<const A*>(p.lora_a) + ((uint64_t)a * p.rank + j) * p.H, p.H * sizeof(A), lane, 32);
    const float scale = a >= 0 ? row_scale(p, t, a) : 0.f;
    for (uint32_t j = warp; j < cols; j += warps) {
        float sum = 0.f;
        if (j < p.rank && a >= 0) {
            const A* row = static_cast<const A*>(p.lora_a) + ((uint64_t)a * p.rank + j) * p.H;
#pragma unroll 4
            for (uint32_t h = lane * 8; h < p.H; h += 256) {
                float xv[8], av[8];
                load_x8(x + h, xv);
                load_x8(row + h, av);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(xv[i], av[i], sum);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            sum = bad ? __int_as_float(0x7fffffff) : sum * scale;
        }
        if (lane == 0) s_u[j] = sum;
    }
    __syncthreads();
    if (warp == 0) write_row(p, t, s_u);
}

// Eight elements of x as four words of the adapters' type (e4m3 values are exact in both).
template <typename A>
__device__ __forceinline__ uint4 load_words(const A* p) { return *reinterpret_cast<const uint4*>(p); }
template <typename A>
__device__ __forceinline__ uint4 load_words(const __nv_fp8_e4m3* p) {
    float v[8];
    load_x8(p, v);
    return make_uint4(pack2(v[0], v[1], A()), pack2(v[2], v[3], A()), pack2(v[4], v[5], A()), pack2(v[6], v[7], A()));
}
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, __nv_bfloat16) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1, __half) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// grid: tiles x ceil(tile_t / 16) blocks of 16 rows, then one a tile for its lists. The 16
// warps split the contraction; their sums are added in the order of the warps.
template <typename X, typename A>
__global__ void __launch_bounds__(kThreads) k_shrink_block(ShrinkParams p) {
    extern __shared__ float s_sum[];              // [kWarps][16][64]
    __shared__ float s_u[kBlockRows][64];
    __shared__ int32_t s_id[kBlockRows];
    pdl_wait();
    pdl_trigger();  // after the wait: the product kernel may read x, which is complete now
    const uint32_t tiles = (p.T + p.tile_t - 1) / p.tile_t, per_tile = p.tile_t / kBlockRows;
    if (blockIdx.x >= tiles * per_tile) {
        list_tile(p, blockIdx.x - tiles * per_tile);
        return;
    }
    const uint32_t tile = blockIdx.x / per_tile, c0 = (blockIdx.x - tile * per_tile) * kBlockRows;
    const uint32_t t0 = tile * p.tile_t + c0;
    if (t0 >= p.T) return;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint32_t cols = rank_cols(p.rank);
    bool bad = false;
    uint32_t code = 0;
    if (threadIdx.x < kBlockRows)
        s_id[threadIdx.x] = t0 + threadIdx.x < p.T ? adapter_of(p, t0 + threadIdx.x, &bad, &code) : -1;
    for (uint32_t i = threadIdx.x; i < kBlockRows * 64; i += kThreads) s_u[i / 64][i % 64] = 0.f;
    __syncthreads();
    const X* x = static_cast<const X*>(p.x);
    const X* xa = x + (uint64_t)min(t0 + g, p.T - 1) * p.x_stride;
    const X* xb = x + (uint64_t)min(t0 + g + 8, p.T - 1) * p.x_stride;
    for (uint32_t r = 0; r < kBlockRows; ++r) {
        const int32_t a = s_id[r];
        bool again = a < 0;  // no adapter, or one of an earlier row
        for (uint32_t i = 0; i < r; ++i) again |= s_id[i] == a;
        if (again) continue;
        float sum[8][4] = {};
        const A* la = static_cast<const A*>(p.lora_a) + (uint64_t)a * p.rank * p.H;
        // 32 terms a step: this thread's are the 8 from h on, the first 4 in one product, the
        // others in the next (their order is the same in both factors)
        uint4 wa, wb, b[8], na, nb, next[8];
        const auto fetch = [&](uint32_t h, uint4& va, uint4& vb, uint4 (&vn)[8]) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
            va = h < p.H ? load_words<A>(xa + h) : zero;
            vb = h < p.H ? load_words<A>(xb + h) : zero;
#pragma unroll
            for (uint32_t n = 0; n < 8; ++n)
                vn[n] = h < p.H && n * 8 + g < p.rank
                            ? *reinterpret_cast<const uint4*>(la + (uint64_t)(n * 8 + g) * p.H + h) : zero;
        };
        uint32_t h = warp * 32 + q * 8;
        fetch(h, wa, wb, b);
        for (; h - q * 8 < p.H; h += kWarps * 32) {
            fetch(h + kWarps * 32, na, nb, next);
#pragma unroll
            for (uint32_t n = 0; n < 8; ++n) {
                if (n * 8 >= p.rank) break;
                mma16(sum[n], wa.x, wb.x, wa.y, wb.y, b[n].x, b[n].y, A());
                mma16(sum[n], wa.z, wb.z, wa.w, wb.w, b[n].z, b[n].w, A());
            }
            wa = na;
            wb = nb;
#pragma unroll
            for (uint32_t n = 0; n < 8; ++n) b[n] = next[n];
        }
        float* mine = s_sum + warp * kBlockRows * 64;
#pragma unroll
        for (uint32_t n = 0; n < 8; ++n) {
            if (n * 8 >= p.rank) break;
            mine[g * 64 + n * 8 + 2 * q] = sum[n][0];
            mine[g * 64 + n * 8 + 2 * q + 1] = sum[n][1];
            mine[(g + 8) * 64 + n * 8 + 2 * q] = sum[n][2];
            mine[(g + 8) * 64 + n * 8 + 2 * q + 1] = sum[n][3];
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < kBlockRows * 64; i += kThreads) {
            const uint32_t row = i / 64, j = i % 64;
            if (s_id[row] != a || j >= p.rank) continue;
            float v = 0.f;
            for (uint32_t w = 0; w < kWarps; ++w) v += s_sum[w * kBlockRows * 64 + i];
            s_u[row][j] = v * row_scale(p, t0 + row, a);
        }
        __syncthreads();
    }
    __syncthreads();
    for (uint32_t row = warp; row < kBlockRows && t0 + row < p.T; row += kWarps) {
        adapter_of(p, t0 + row, &bad, &code);
        if (bad) {
            if (lane == 0) flag(p.status, code);
            for (uint32_t j = lane; j < cols; j += 32) s_u[row][j] = __int_as_float(0x7fffffff);
            __syncwarp();
        }
        write_row(p, t0 + row, s_u[row]);
    }
}

template <typename X, typename A>
lp_status launch_shrink(const ShrinkParams& p, lp_stream_t s) {
    const uint32_t tiles = (p.T + p.tile_t - 1) / p.tile_t;
    // A block of 16 rows takes its adapters one after the other, a row a block its rank's dot
    // products. Whole projections onto 512 tokens, us (blocks | rows), H = 4096, rank 16 and 64:
    //     77 rows, 4 a request  50 | 32, 66 | 38    16 a request  31 | 29, 33 | 33
    //    256 rows, 4 a request  50 | 40, 64 | 51     8 a request  36 | 38, 44 | 47
    //   1024 rows, 2 a request  77 | 56, 101 | 107   4 a request  52 | 54, 66 | 105
    const uint32_t sms = (uint32_t)sm_count(), rows_a_request = p.T / p.B;
    if (p.T > sms && rows_a_request >= (p.T > 2 * sms ? 4u : 8u)) {
        static std::atomic<uint64_t> smem_set;
        if (!allow_smem(reinterpret_cast<const void*>(k_shrink_block<X, A>), kWarps * kBlockRows * 64 * sizeof(float),
                        &smem_set))
            return LP_ERR_CUDA;
        return launch(k_shrink_block<X, A>, dim3(tiles * (p.tile_t / kBlockRows) + tiles), kThreads,
                      kWarps * kBlockRows * 64 * sizeof(float), s, 1, p);
    }
    // a warp a dot product, up to 16; the lists take kMaxTileT threads
    const uint32_t warps = rank_cols(p.rank) < 16 ? 16 : rank_cols(p.rank) > 32 ? 32 : rank_cols(p.rank);
    return launch(k_shrink_row<X, A>, dim3(p.T + tiles), warps * 32, 0, s, 1, p);
}

}  // namespace

namespace lph {

lp_status launch_shrink(const ShrinkParams& p, uint32_t dtype, uint32_t lora_dtype, lp_stream_t s) {
    if (dtype == LP_BF16) return ::launch_shrink<__nv_bfloat16, __nv_bfloat16>(p, s);
    if (dtype == LP_F16) return ::launch_shrink<__half, __half>(p, s);
    if (lora_dtype == LP_BF16) return ::launch_shrink<__nv_fp8_e4m3, __nv_bfloat16>(p, s);
    return ::launch_shrink<__nv_fp8_e4m3, __half>(p, s);
}

}  // namespace lph

extern "C" size_t lp_head_workspace_size(uint32_t T, uint32_t rank) {
    return rank > LP_MAX_RANK ? 0 : lph::AdapterSpace(T, rank).bytes;
}
