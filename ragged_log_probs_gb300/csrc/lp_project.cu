// Projection of hidden states to logits with low-rank adapters (include/lp_head.h):
//     out[t, v] = sx[t] sw[v] sum_h x[t, h] W[v, h] + sum_j u[t, j] B_a[v, j],
//     u[t, j]   = s_a sx[t] sum_h x[t, h] A_a[j, h],   a = adapter of row t's request.
//
// The product runs on the tensor cores with the vocabulary on the accumulator's lanes: a
// tile is 128 vocabulary rows by N rows of x (N = the row count rounded up to 16, at most
// 256), so that a decode step reads W once and pads little, and a warp's 32 lanes hold 32
// neighbouring logits of one output row (coalesced stores without a transpose). One thread
// issues TMA copies of 128-byte-wide slices of W and x into a ring of stages, one issues
// tcgen05.mma from them into one of two accumulators in TMEM, and eight warps empty the
// other accumulator meanwhile. Kernels are persistent; consecutive tiles share their W rows.
//
// u is computed first, by its own small kernel; the product starts while that still runs
// and waits for it only before its first epilogue, which adds the adapters' part in f32.
#include <cuda.h>

#include "lp_head_common.h"

namespace {

using namespace lph;

constexpr uint32_t kTileV = 128;                  // vocabulary rows of a tile (accumulator lanes)
constexpr uint32_t kMaxTileT = 256;               // rows of x of a tile
constexpr uint32_t kSliceBytes = 128;             // bytes of the contracted dimension per stage
constexpr uint32_t kStageW = kTileV * kSliceBytes;
constexpr uint32_t kMaxStages = 12;
constexpr uint32_t kEpilogueWarps = 8;
constexpr uint32_t kFirstEpilogueWarp = 4;
constexpr uint32_t kThreads = (kFirstEpilogueWarp + kEpilogueWarps) * 32;
constexpr uint32_t kSmemBudget = 227 * 1024;
constexpr uint32_t kControlBytes = 1024 + 256;    // barriers and words, and the alignment of the ring

struct ProjectParams {
    const float* x_scale;
    const float* w_scale;
    const void* lora_b;      // [A][V][rank]
    const float* u;          // [T][rank]
    const int32_t* ids;      // [T] adapter of each row, negative: none
    void* out;
    uint32_t* status;
    uint64_t out_stride;
    uint32_t T, V, rank;
    uint32_t tile_t;         // N
    uint32_t tiles_t, tiles, slices, stages;
    uint32_t acc_cols;       // TMEM columns of one accumulator
    uint32_t idesc;
    uint32_t lora_f16;       // lora_b is f16 (else bf16)
    uint32_t early;          // the inputs are complete when this kernel starts (u may not be)
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}
// Every wait ends: after kWaitNs the CTA's abort word is set, and every role that sees it
// gives up (the host reads LP_ERR_TIMEOUT).
constexpr uint64_t kWaitNs = 2000000000ull;
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_word) {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = now_ns();
    for (uint32_t n = 0; n < (1u << 30); ++n) {
        if (mbar_try(bar, parity)) return true;
        if (*abort_word) return false;
        if (now_ns() - t0 > kWaitNs) break;
    }
    *abort_word = 1;
    return false;
}

// The same for a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile uint32_t* abort_word) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_word));
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar), "l"(policy) : "memory");
}

// Shared-memory matrix descriptor: rows of 128 bytes, 128-byte swizzle, groups of 8 rows
// 1024 bytes apart, contracted dimension contiguous.
__device__ __forceinline__ uint64_t matrix_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <bool FP8>
__device__ __forceinline__ void mma(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (FP8)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem), "l"(a), "l"(b),
                     "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem), "l"(a), "l"(b),
                     "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr) : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Sixteen values of row v of an adapter's B, from j0 on (zero past the rank).
__device__ __forceinline__ void load_b(const ProjectParams& p, uint32_t a, uint32_t v, uint32_t j0, float (&b)[16]) {
    const uint16_t* row = static_cast<const uint16_t*>(p.lora_b) + ((uint64_t)a * p.V + v) * p.rank + j0;
    const uint32_t left = p.rank - j0;
    uint32_t w[8];
    if (left >= 16 && p.rank % 8 == 0) {
        const uint4 lo = *reinterpret_cast<const uint4*>(row), hi = *reinterpret_cast<const uint4*>(row + 8);
        w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
        w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t l = 2 * i < left ? row[2 * i] : 0u, h = 2 * i + 1 < left ? row[2 * i + 1] : 0u;
            w[i] = l | (h << 16);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = p.lora_f16 ? unpack2(w[i], __half()) : unpack2(w[i], __nv_bfloat16());
        b[2 * i] = f.x;
        b[2 * i + 1] = f.y;
    }
}

template <bool FP8, typename OUT>
__global__ void __launch_bounds__(kThreads, 1)
k_project(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const ProjectParams p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* ring = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t N = p.tile_t, stage_bytes = kStageW + N * kSliceBytes;
    const uint32_t rp = (p.rank + 15) & ~15u;  // rank, padded with zeros
    float* s_u = reinterpret_cast<float*>(ring + p.stages * stage_bytes);       // [N][rp]
    float* s_scale = s_u + N * rp;                                              // [N]
    int32_t* s_id = reinterpret_cast<int32_t*>(s_scale + N);                    // [N]
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_id + N);
    volatile uint32_t* s_abort = reinterpret_cast<uint32_t*>(bars + 2 * kMaxStages + 6);
    uint32_t* s_tmem = const_cast<uint32_t*>(s_abort) + 1;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages, acc_full0 = empty0 + 8 * kMaxStages,
                   acc_empty0 = acc_full0 + 16, drain = acc_empty0 + 16, staging = drain + 8;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < p.stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(acc_full0 + 8 * i, 1);
            mbar_init(acc_empty0 + 8 * i, kEpilogueWarps);
        }
        mbar_init(drain, 1);
        mbar_init(staging, kEpilogueWarps);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                     "r"(2 * p.acc_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *s_tmem;

    uint32_t issued = 0;  // stages the producer has started copies into
    if (warp == 0) {
        if (lane == 0) {
            if (!p.early) pdl_wait();
            uint64_t once, keep;  // W is read once per row of tiles, x by every tile
            asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
            asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
            const uint64_t w_policy = p.tiles_t == 1 ? once : keep;
            const uint32_t slice_elems = FP8 ? kSliceBytes : kSliceBytes / 2;
            uint32_t s = 0, phase = 0;
            bool ok = true;
            for (uint32_t tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x) {
                const uint32_t tv = tile / p.tiles_t, tt = tile - tv * p.tiles_t;
                for (uint32_t k = 0; k < p.slices; ++k) {
                    if (!mbar_wait(empty0 + 8 * s, phase ^ 1, s_abort)) { ok = false; break; }
                    const uint32_t dst = base + s * stage_bytes, bar = full0 + 8 * s;
                    mbar_expect(bar, stage_bytes);
                    tma_2d(dst, &map_w, (int)(k * slice_elems), (int)(tv * kTileV), bar, w_policy);
                    tma_2d(dst + kStageW, &map_x, (int)(k * slice_elems), (int)(tt * N), bar, keep);
                    ++issued;
                    if (++s == p.stages) { s = 0; phase ^= 1; }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t s = 0, phase = 0, n = 0;
            bool ok = true;
            for (uint32_t tile = blockIdx.x; ok && tile < p.tiles; tile += gridDim.x, ++n) {
                const uint32_t acc = n & 1, acc_phase = (n >> 1) & 1;
                if (!mbar_wait(acc_empty0 + 8 * acc, acc_phase ^ 1, s_abort)) break;
                fence_after();
                for (uint32_t k = 0; k < p.slices; ++k) {
                    if (!mbar_wait(full0 + 8 * s, phase, s_abort)) { ok = false; break; }
                    fence_after();
                    const uint64_t a = matrix_desc(base + s * stage_bytes);
                    const uint64_t b = matrix_desc(base + s * stage_bytes + kStageW);
#pragma unroll
                    for (uint32_t i = 0; i < kSliceBytes / 32; ++i)  // 32 bytes of the contracted dimension each
                        mma<FP8>(tmem + acc * p.acc_cols, a + 2 * i, b + 2 * i, p.idesc, k | i);
                    mma_commit(empty0 + 8 * s);
                    if (++s == p.stages) { s = 0; phase ^= 1; }
                }
                if (ok) mma_commit(acc_full0 + 8 * acc);
            }
            mma_commit(drain);  // arrives once every product issued above has finished
        }
    } else if (warp >= kFirstEpilogueWarp) {
        // Quadrant of lanes this warp may read, and which 32-column groups it takes.
        const uint32_t quad = warp & 3, half = (warp - kFirstEpilogueWarp) >> 2;
        const uint32_t et = threadIdx.x - kFirstEpilogueWarp * 32;
        OUT* out = static_cast<OUT*>(p.out);
        uint32_t n = 0, staged = 0xFFFFFFFFu, staging_phase = 0;
        // all epilogue warps have come here (a bounded wait, as everywhere: no warp can be
        // left behind by one that gave up)
        const auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(staging);
            const bool ok = mbar_wait_warp(staging, staging_phase, s_abort);
            staging_phase ^= 1;
            return ok;
        };
        pdl_wait();
        for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, ++n) {
            const uint32_t acc = n & 1, acc_phase = (n >> 1) & 1;
            const uint32_t tv = tile / p.tiles_t, tt = tile - tv * p.tiles_t, t0 = tt * N;
            const uint32_t v = tv * kTileV + quad * 32 + lane;
            if (tt != staged) {  // the rows' adapters, u and scales
                if (!meet()) break;
                for (uint32_t i = et; i < N; i += kEpilogueWarps * 32) {
                    s_id[i] = p.rank && t0 + i < p.T ? p.ids[t0 + i] : -1;
                    s_scale[i] = FP8 && t0 + i < p.T ? p.x_scale[t0 + i] : 1.f;
                }
                for (uint32_t i = et; i < N * rp; i += kEpilogueWarps * 32) {
                    const uint32_t c = i / rp, j = i - c * rp;
                    s_u[i] = t0 + c < p.T && j < p.rank ? p.u[(uint64_t)(t0 + c) * p.rank + j] : 0.f;
                }
                if (!meet()) break;
                staged = tt;
            }
            const float sw = FP8 && v < p.V ? p.w_scale[v] : 1.f;
            if (!mbar_wait_warp(acc_full0 + 8 * acc, acc_phase, s_abort)) break;
            fence_after();
            for (uint32_t c0 = half * 32; c0 < N; c0 += 64) {
                float y[32];
                tmem_load32(tmem + ((quad * 32) << 16) + acc * p.acc_cols + c0, y);
                if constexpr (FP8) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) y[c] *= sw * (c0 + c < N ? s_scale[c0 + c] : 0.f);
                }
                if (p.rank) {
                    const int32_t id = c0 + lane < N ? s_id[c0 + lane] : -1;
                    uint32_t todo = __ballot_sync(0xFFFFFFFFu, id >= 0);
                    while (todo) {  // the group's rows of one adapter together
                        const int32_t a = __shfl_sync(0xFFFFFFFFu, id, __ffs(todo) - 1);
                        const uint32_t mine = __ballot_sync(0xFFFFFFFFu, id == a);
                        todo &= ~mine;
                        for (uint32_t j0 = 0; j0 < rp; j0 += 16) {
                            float b[16];
                            load_b(p, (uint32_t)a, v < p.V ? v : p.V - 1, j0, b);
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                if (mine >> c & 1) {
                                    const float4* u4 = reinterpret_cast<const float4*>(s_u + (c0 + c) * rp + j0);
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        const float4 u = u4[i];
                                        y[c] = fmaf(u.x, b[4 * i], y[c]);
                                        y[c] = fmaf(u.y, b[4 * i + 1], y[c]);
                                        y[c] = fmaf(u.z, b[4 * i + 2], y[c]);
                                        y[c] = fmaf(u.w, b[4 * i + 3], y[c]);
                                    }
                                }
                            }
                        }
                    }
                }
                if (v < p.V) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (c0 + c < N && t0 + c0 + c < p.T)
                            out[(uint64_t)(t0 + c0 + c) * p.out_stride + v] = from_f32<OUT>(y[c]);
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty0 + 8 * acc);
        }
    }
    // Everything issued is finished before shared memory and TMEM go: in a normal run the
    // epilogue has seen every tile; after an abort the copies and products in flight end by
    // themselves, and these waits are bounded like the others.
    if (warp == 1 && lane == 0) {
        uint32_t dummy = 0;
        (void)mbar_wait(drain, 0, &dummy);
    }
    if (warp == 0 && lane == 0 && *s_abort) {
        for (uint32_t i = issued < p.stages ? 0 : issued - p.stages; i < issued; ++i) {
            uint32_t dummy = 0;
            (void)mbar_wait(full0 + 8 * (i % p.stages), (i / p.stages) & 1, &dummy);
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * p.acc_cols));
    if (threadIdx.x == 0 && *s_abort) flag(p.status, LP_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ u = s_a sx (x A_a^T)

struct ShrinkParams {
    const void* x;
    const float* x_scale;
    const void* lora_a;            // [A][rank][H]
    const float* adapter_scale;    // [A] or NULL
    const int32_t* adapter_ids;    // [B]
    const uint32_t* row_offsets;   // [B+1] or NULL
    float* u;
    int32_t* ids;
    uint32_t* status;
    uint64_t x_stride;
    uint32_t T, H, B, adapters, rank;
};

constexpr uint32_t kShrinkWarps = 8;

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

template <typename X, typename A>
__global__ void __launch_bounds__(kShrinkWarps * 32) k_shrink(ShrinkParams p) {
    pdl_wait();
    pdl_trigger();  // after the wait: the product kernel may read x, which is complete now
    const uint32_t t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = request_of(p.row_offsets, p.B, t);
    int32_t a = b < 0 ? 0 : p.adapter_ids[b];
    const bool bad = b < 0 || a >= (int32_t)p.adapters;
    if (bad) {
        a = 0;
        if (threadIdx.x == 0) flag(p.status, b < 0 ? LP_ERR_OFFSETS : LP_ERR_ADAPTER);
    }
    if (threadIdx.x == 0) p.ids[t] = a;
    if (a < 0) return;
    const X* x = static_cast<const X*>(p.x) + (uint64_t)t * p.x_stride;
    float scale = p.adapter_scale ? p.adapter_scale[a] : 1.f;
    if (p.x_scale) scale *= p.x_scale[t];
    for (uint32_t j = warp; j < p.rank; j += kShrinkWarps) {
        const A* row = static_cast<const A*>(p.lora_a) + ((uint64_t)a * p.rank + j) * p.H;
        float sum = 0.f;
        for (uint32_t h = lane * 8; h < p.H; h += 256) {
            float xv[8], av[8];
            load_x8(x + h, xv);
            load_x8(row + h, av);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(xv[i], av[i], sum);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (lane == 0) p.u[(uint64_t)t * p.rank + j] = bad ? __int_as_float(0x7fffffff) : sum * scale;
    }
}

// ------------------------------------------------------------------ host

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static std::atomic<EncodeFn> known{nullptr};
    EncodeFn f = known.load(std::memory_order_acquire);
    if (!f) {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &found) !=
                cudaSuccess || found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return nullptr;
        }
        f = reinterpret_cast<EncodeFn>(ptr);
        known.store(f, std::memory_order_release);
    }
    return f;
}

// Map of a row-major matrix [rows][cols], read in boxes of 128 bytes by box_rows rows.
bool encode(CUtensorMap* map, const void* ptr, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t stride,
            uint32_t box_rows) {
    const EncodeFn f = encode_fn();
    if (!f) return false;
    const CUtensorMapDataType type = dtype == LP_E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : dtype == LP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t e = dtype_bytes(dtype);
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {stride * e};
    const cuuint32_t box[2] = {(cuuint32_t)(kSliceBytes / e), box_rows}, step[2] = {1, 1};
    return f(map, type, 2, const_cast<void*>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

std::atomic<uint64_t> g_smem_set[2][3];

template <bool FP8, typename OUT>
lp_status launch_project(const CUtensorMap& w, const CUtensorMap& x, const ProjectParams& p, unsigned grid, size_t smem,
                         int out_index, lp_stream_t stream) {
    auto kernel = k_project<FP8, OUT>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), kSmemBudget, &g_smem_set[FP8][out_index])) return LP_ERR_CUDA;
    return launch(kernel, dim3(grid), kThreads, smem, stream, 1, w, x, p);
}

template <bool FP8>
lp_status launch_project(const CUtensorMap& w, const CUtensorMap& x, const ProjectParams& p, unsigned grid, size_t smem,
                         uint32_t out_dtype, lp_stream_t stream) {
    if (out_dtype == LP_F32) return launch_project<FP8, float>(w, x, p, grid, smem, 0, stream);
    if (out_dtype == LP_BF16) return launch_project<FP8, __nv_bfloat16>(w, x, p, grid, smem, 1, stream);
    return launch_project<FP8, __half>(w, x, p, grid, smem, 2, stream);
}

lp_status launch_shrink(const ShrinkParams& p, uint32_t dtype, uint32_t lora_dtype, lp_stream_t s) {
    const dim3 grid(p.T);
    const unsigned block = kShrinkWarps * 32;
    if (dtype == LP_BF16) return launch(k_shrink<__nv_bfloat16, __nv_bfloat16>, grid, block, 0, s, 1, p);
    if (dtype == LP_F16) return launch(k_shrink<__half, __half>, grid, block, 0, s, 1, p);
    if (lora_dtype == LP_BF16) return launch(k_shrink<__nv_fp8_e4m3, __nv_bfloat16>, grid, block, 0, s, 1, p);
    return launch(k_shrink<__nv_fp8_e4m3, __half>, grid, block, 0, s, 1, p);
}

}  // namespace

extern "C" lp_status lp_head_project(const void* x, uint32_t dtype, uint32_t T, uint32_t H, uint64_t x_stride,
                                     const float* x_scale, const void* weight, uint32_t V, uint64_t weight_stride,
                                     const float* weight_scale, const void* lora_a, const void* lora_b,
                                     uint32_t lora_dtype, uint32_t adapters, uint32_t rank,
                                     const float* adapter_scale, const int32_t* adapter_ids,
                                     const uint32_t* row_offsets, uint32_t B, void* out, uint32_t out_dtype,
                                     uint64_t out_stride, void* workspace, size_t workspace_bytes,
                                     lp_stream_t stream) {
    if (!x || !weight || !out) return LP_ERR_NULL;
    if (dtype != LP_BF16 && dtype != LP_F16 && dtype != LP_E4M3) return LP_ERR_DTYPE;
    if (out_dtype != LP_F32 && out_dtype != LP_BF16 && out_dtype != LP_F16) return LP_ERR_DTYPE;
    const bool fp8 = dtype == LP_E4M3, adapted = adapters != 0;
    if (fp8 && (!x_scale || !weight_scale)) return LP_ERR_NULL;
    if (!fp8 && (x_scale || weight_scale)) return LP_ERR_DTYPE;
    if (T == 0 || H == 0 || V == 0 || T > 0x7FFFFF00u || V > 0x7FFFFF00u || H > 0x7FFFFF00u) return LP_ERR_SHAPE;
    if (x_stride < H || weight_stride < H || out_stride < V) return LP_ERR_SHAPE;
    const size_t e = dtype_bytes(dtype), eo = dtype_bytes(out_dtype);
    // the copies start on 16-byte boundaries and move whole 16 bytes
    if (!aligned_to(x, 16) || !aligned_to(weight, 16) || H * e % 16 || x_stride * e % 16 || weight_stride * e % 16)
        return LP_ERR_SHAPE;
    if (!aligned_to(out, eo) || !aligned_to(x_scale, 4) || !aligned_to(weight_scale, 4)) return LP_ERR_SHAPE;
    if (adapted) {
        if (!lora_a || !lora_b || !adapter_ids) return LP_ERR_NULL;
        if (rank == 0 || rank > LP_MAX_RANK || adapters > 0x7FFFFFFFu) return LP_ERR_SHAPE;
        if (lora_dtype != LP_BF16 && lora_dtype != LP_F16) return LP_ERR_DTYPE;
        if (!fp8 && lora_dtype != dtype) return LP_ERR_DTYPE;
        if (B == 0 || (!row_offsets && B != T)) return LP_ERR_SHAPE;
        if (!aligned_to(lora_a, 16) || !aligned_to(lora_b, 16)) return LP_ERR_SHAPE;
    } else {
        rank = 0;
    }
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < lp_head_workspace_size(rank ? T : 0, rank))
        return LP_ERR_WORKSPACE;
    const int sms = sm_count();
    if (sms == 0) return LP_ERR_CUDA;

    unsigned char* ws = static_cast<unsigned char*>(workspace);
    ProjectParams p = {};
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.x_scale = x_scale;
    p.w_scale = weight_scale;
    p.lora_b = lora_b;
    p.ids = reinterpret_cast<int32_t*>(ws + kHeaderBytes);
    p.u = reinterpret_cast<float*>(ws + kHeaderBytes + (((size_t)T * 4 + 255) & ~(size_t)255));
    p.out = out;
    p.out_stride = out_stride;
    p.T = T;
    p.V = V;
    p.rank = rank;
    p.lora_f16 = lora_dtype == LP_F16;
    p.early = rank != 0;
    // Rows of x in even tiles of at most 256, a multiple of 16.
    p.tiles_t = (T + kMaxTileT - 1) / kMaxTileT;
    p.tile_t = ((T + p.tiles_t - 1) / p.tiles_t + 15) & ~15u;
    const uint64_t tiles = (uint64_t)((V + kTileV - 1) / kTileV) * p.tiles_t;
    if (tiles > 0x7FFFFFFFu) return LP_ERR_SHAPE;
    p.tiles = (uint32_t)tiles;
    p.slices = (uint32_t)((H * e + kSliceBytes - 1) / kSliceBytes);
    for (p.acc_cols = 32; p.acc_cols < p.tile_t; p.acc_cols *= 2) {}
    // instruction: f32 accumulator, K-major operands, M = 128, N = tile_t
    const uint32_t type = dtype == LP_BF16 ? 1u : 0u;  // kind::f16: 0 f16, 1 bf16; kind::f8f6f4: 0 e4m3
    p.idesc = (1u << 4) | (type << 7) | (type << 10) | ((p.tile_t >> 3) << 17) | ((kTileV >> 4) << 24);
    const uint32_t rp = (rank + 15) & ~15u, stage_bytes = kStageW + p.tile_t * kSliceBytes;
    const uint32_t rows_bytes = p.tile_t * (rp * 4 + 8);
    p.stages = (kSmemBudget - kControlBytes - rows_bytes) / stage_bytes;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    const size_t smem = kControlBytes + rows_bytes + p.stages * stage_bytes;
    CUtensorMap map_w, map_x;
    if (!encode(&map_w, weight, dtype, V, H, weight_stride, kTileV) ||
        !encode(&map_x, x, dtype, T, H, x_stride, p.tile_t))
        return LP_ERR_CUDA;
    if (rank) {
        ShrinkParams q = {};
        q.x = x;
        q.x_scale = x_scale;
        q.lora_a = lora_a;
        q.adapter_scale = adapter_scale;
        q.adapter_ids = adapter_ids;
        q.row_offsets = row_offsets;
        q.u = const_cast<float*>(p.u);
        q.ids = const_cast<int32_t*>(p.ids);
        q.status = p.status;
        q.x_stride = x_stride;
        q.T = T;
        q.H = H;
        q.B = B;
        q.adapters = adapters;
        q.rank = rank;
        const lp_status st = launch_shrink(q, dtype, lora_dtype, stream);
        if (st != LP_OK) return st;
    }
    const unsigned grid = p.tiles < (uint32_t)sms ? p.tiles : (unsigned)sms;
    return fp8 ? launch_project<true>(map_w, map_x, p, grid, smem, out_dtype, stream)
               : launch_project<false>(map_w, map_x, p, grid, smem, out_dtype, stream);
}
