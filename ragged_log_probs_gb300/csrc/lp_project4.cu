// Projection of microscaled 4-bit hidden states to logits (include/lp_head.h):
//     out[t, v] = sx[t] sw[v] sum_b X_b[t] W_b[v] sum_{h in b} x[t, h] w[v, h]
// with x, w in e2m1 and one scale for every block b of 16 (e4m3) or 32 (e8m0) elements.
//
// The tensor cores multiply such blocks with their scales. As in the projection of wider types the
// vocabulary lies on the accumulator's lanes: a tile is 128 vocabulary rows (256 of a pair of
// CTAs) by N rows of x, one thread issues TMA copies of 128-byte-wide slices (256 elements) of W
// and x and of their scales into a ring of stages, one issues the products, and twelve warps
// empty the accumulators. The scales go from a stage through tcgen05.cp into TMEM, where the
// products read them; each stage of the ring has columns of its own there, so that they are
// written again only after the products that read them have been waited for. 256 columns hold
// the accumulators (two of 128, or one), 256 the scales. The epilogue takes a finished
// accumulator into registers at once and hands it back before it stores.
//
// Few rows are bound by HBM: 48 on V = 152064, H = 4096 66 us (350 MB of W and scales in 5.8 TB/s, 86 %
// of a copy's rate). Many rows are bound by the tensor cores: 2048 on 32000 x 4096 91 us (5.9 PFLOP/s, the
// pipe active 65 % of the time); a further 4096 of H cost 64 us (8.3 PFLOP/s), the rest is the start, the
// last wave of tiles, and 1.2 us a tile for which the one accumulator of 256 columns is being
// emptied. Loads of all columns before one wait for them were not faster.
#include "lp_tcgen05.h"

namespace {

using namespace lph;

constexpr uint32_t kTileV = 128;
constexpr uint32_t kSliceBytes = 128;    // 256 elements
constexpr uint32_t kSlice = 256;
constexpr uint32_t kStageW = kTileV * kSliceBytes;
constexpr uint32_t kMaxTileT = 256;
constexpr uint32_t kMaxStages = 8;
constexpr uint32_t kEpilogueWarps = 12;
constexpr uint32_t kShares = kEpilogueWarps / 4;
constexpr uint32_t kMaxBlocks = (kMaxTileT / 32 + kShares - 1) / kShares;  // of 32 columns, of an epilogue warp
constexpr uint32_t kCopyWarp = kEpilogueWarps, kMmaWarp = kEpilogueWarps + 1;
constexpr uint32_t kThreads = (kEpilogueWarps + 2) * 32;
constexpr uint32_t kControlBytes = 1024 + 256;
constexpr uint32_t kColumns = 512, kScaleColumns = 256;  // of TMEM; where the scales begin

struct Project4Params {
    const float* x_scale;  // [T] or NULL
    const float* w_scale;  // [V] or NULL
    void* out;
    uint32_t* status;
    uint64_t out_stride;
    uint32_t T, V, H;
    uint32_t tile_t, tiles_t, tiles, slices, stages;
    uint32_t col_tiles;    // tiles of scales in a row of them
    uint32_t acc_shift;    // log2 of the number of accumulators
    uint32_t idesc;        // without N and the scales' places
};

constexpr uint32_t kBarriers = 2 * kMaxStages + 4 + 1;

// Shared-memory descriptor of a tile of scales: 32 rows of 16 bytes, no swizzle.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
}
// A tile of scales into four columns, the same for all four quadrants of lanes (of both CTAs of a
// pair, each from its own shared memory).
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    if constexpr (CG == 2) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
template <int BLOCK, int CG>
__device__ __forceinline__ void mma4(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                     uint32_t accumulate) {
#define LPH_MMA4(GROUP, KIND)                                                                            \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"                                     \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" \
                 ::"r"(tmem), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) : "memory")
    if constexpr (BLOCK == 16 && CG == 2) LPH_MMA4("2", "mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (BLOCK == 16) LPH_MMA4("1", "mxf4nvf4.block_scale.scale_vec::4X");
    else if constexpr (CG == 2) LPH_MMA4("2", "mxf4.block_scale.scale_vec::2X");
    else LPH_MMA4("1", "mxf4.block_scale.scale_vec::2X");
#undef LPH_MMA4
}

__device__ __forceinline__ bool elect_one() {  // the same lane of a whole warp every time
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

template <int BLOCK, typename OUT, int CG>
__global__ void __launch_bounds__(kThreads, 1)
k_project4(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
           const __grid_constant__ CUtensorMap map_ws, const __grid_constant__ CUtensorMap map_xs, const Project4Params p) {
    // tiles of scales in a slice: 4 blocks of 16 or 32 elements each
    constexpr uint32_t kTiles = kSlice / (4 * BLOCK), kScaleBytes = kTiles * 512;
    constexpr uint32_t kXBlocks = CG;  // blocks of 128 rows of x in a tile
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t stage_x = p.tile_t / CG * kSliceBytes;
    const uint32_t stage_bytes = kStageW + stage_x + (1 + kXBlocks) * kScaleBytes;
    unsigned char* ring = smem_raw + (base - smem_u32(smem_raw));
    uint64_t* bars = reinterpret_cast<uint64_t*>(ring + p.stages * stage_bytes);
    volatile uint32_t* s_abort = reinterpret_cast<uint32_t*>(bars + kBarriers);
    uint32_t* s_tmem = const_cast<uint32_t*>(s_abort) + 1;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages, acc_full0 = empty0 + 8 * kMaxStages,
                   acc_empty0 = acc_full0 + 16, drain = acc_empty0 + 16;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank = 0;
    if constexpr (CG == 2) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const uint32_t first = blockIdx.x / CG, step = gridDim.x / CG;
    const auto acc_of = [&](uint32_t n) { return n & ((1u << p.acc_shift) - 1); };
    const auto acc_phase = [&](uint32_t n) { return n >> p.acc_shift & 1; };
    // rows of x in tile tt, a whole number of 16 for each CTA
    const auto rows_of = [&](uint32_t tt) { return min(p.tile_t, (p.T - tt * p.tile_t + 16 * CG - 1) / (16 * CG) * (16 * CG)); };

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < p.stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(acc_full0 + 8 * i, 1);
            mbar_init(acc_empty0 + 8 * i, kEpilogueWarps * CG);
        }
        mbar_init(drain, 1);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        if constexpr (CG == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                         "r"(kColumns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                         "r"(kColumns) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();  // the other CTA's barriers are ready too
    fence_after();
    const uint32_t tmem = *s_tmem;

    uint32_t issued = 0;  // stages the producer has started copies into
    if (warp == kCopyWarp) {
        pdl_wait();
        uint64_t once, keep;  // W is read once per row of tiles, x by every tile
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
        const uint64_t w_policy = p.tiles_t == 1 ? once : keep;
        const uint32_t w_blocks = (p.V + 127) / 128, all_x_blocks = (p.T + 127) / 128;
        const bool elected = elect_one();
        uint32_t s = 0, phase = 0;
        bool ok = true;
        for (uint32_t tile = first; ok && tile < p.tiles; tile += step) {
            const uint32_t tv = tile / p.tiles_t, tt = tile - tv * p.tiles_t;
            const uint32_t block = tv * CG + rank, n = rows_of(tt);
            const int v0 = (int)(block * kTileV), t0 = (int)(tt * p.tile_t + rank * (n / CG));
            // (scales of blocks of 128 rows past the last: any, their products are not stored)
            const uint32_t ws_row = min(block, w_blocks - 1) * p.col_tiles;
            uint32_t xs_row[kXBlocks];
#pragma unroll
            for (uint32_t j = 0; j < kXBlocks; ++j) xs_row[j] = min(tt * kXBlocks + j, all_x_blocks - 1) * p.col_tiles;
            for (uint32_t k = 0; k < p.slices; ++k) {
                if (!mbar_wait_warp(empty0 + 8 * s, phase ^ 1, s_abort)) { ok = false; break; }
                if (elected) {
                    const uint32_t dst = base + s * stage_bytes;
                    const uint32_t bar = CG == 2 ? map_to(full0 + 8 * s, 0) : full0 + 8 * s;
                    if (rank == 0) mbar_expect(full0 + 8 * s, CG * stage_bytes);
                    tma_2d<CG>(dst, &map_w, (int)(k * kSliceBytes), v0, bar, w_policy);
                    tma_2d<CG>(dst + kStageW + stage_x, &map_ws, 0, (int)(ws_row + k * kTiles), bar, w_policy);
                    tma_2d<CG>(dst + kStageW, &map_x, (int)(k * kSliceBytes), t0, bar, keep);
#pragma unroll
                    for (uint32_t j = 0; j < kXBlocks; ++j)
                        tma_2d<CG>(dst + kStageW + stage_x + (1 + j) * kScaleBytes, &map_xs, 0,
                                   (int)(xs_row[j] + k * kTiles), bar, keep);
                }
                __syncwarp();
                ++issued;
                if (++s == p.stages) { s = 0; phase ^= 1; }
            }
        }
    } else if (warp == kMmaWarp) {
        // The whole warp walks the tiles, so that what the instructions take is known to be the same
        // for its lanes, and an elected one issues them: 8 clocks a copy of scales, against 50 to 180
        // from a branch of lane 0 (48 rows on V = 152064: 116 us so).
        if (rank == 0) {
            pdl_wait();  // (the bounded waits below are for this kernel's own work only)
            constexpr uint32_t kSlot = kTiles * 4 * (1 + kXBlocks);  // columns of a stage's scales
            const bool elected = elect_one();
            uint32_t s = 0, phase = 0, n = 0;
            bool ok = true;
            for (uint32_t tile = first; ok && tile < p.tiles; tile += step) {
                const uint32_t idesc = p.idesc | ((rows_of(tile % p.tiles_t) >> 3) << 17);
                const uint32_t acc = acc_of(n), d = tmem + acc * (kMaxTileT / 2);
                if (!mbar_wait_warp(acc_empty0 + 8 * acc, acc_phase(n) ^ 1, s_abort)) { ok = false; break; }
                fence_after();
                for (uint32_t k = 0; k < p.slices; ++k) {
                    if (!mbar_wait_warp(full0 + 8 * s, phase, s_abort)) { ok = false; break; }
                    fence_after();
                    const uint32_t at = base + s * stage_bytes, scales = at + kStageW + stage_x;
                    const uint64_t a = matrix_desc(at), b = matrix_desc(at + kStageW), c = scale_desc(scales);
                    const uint32_t sa = tmem + kScaleColumns + s * kSlot, sb = sa + kTiles * 4;
                    const uint32_t steps = min(4u, (p.H - k * kSlice + 63) / 64);  // of 64 elements
                    if (elected) {
#pragma unroll
                        for (uint32_t j = 0; j < kTiles; ++j) {
                            copy_scales<CG>(sa + 4 * j, c + j * (512 >> 4));
#pragma unroll
                            for (uint32_t q = 0; q < kXBlocks; ++q)
                                copy_scales<CG>(sb + 4 * (kXBlocks * j + q), c + ((1 + q) * kScaleBytes + j * 512 >> 4));
                        }
#pragma unroll
                        for (uint32_t i = 0; i < 4; ++i) {
                            // blocks of 32: a tile's columns hold the scales of two steps
                            const uint32_t j = BLOCK == 16 ? i : i / 2, id = BLOCK == 16 ? 0 : (i & 1) * 2;
                            if (i < steps)
                                mma4<BLOCK, CG>(d, a + 2 * i, b + 2 * i, idesc | id << 4 | id << 29, sa + 4 * j,
                                                sb + 4 * kXBlocks * j, k | i);
                        }
                        mma_commit<CG>(empty0 + 8 * s);
                    }
                    __syncwarp();
                    if (++s == p.stages) { s = 0; phase ^= 1; }
                }
                if (!ok) break;
                if (elected) mma_commit<CG>(acc_full0 + 8 * acc);
                ++n;
            }
            if (elected) mma_commit<CG>(drain);  // arrives once every product issued above has finished
            __syncwarp();
        }
    } else {
        // The quadrant of lanes this warp may read, and its share of the columns: the blocks
        // of 32 whose number is `share` modulo kShares.
        const uint32_t quad = warp & 3, share = warp >> 2;
        OUT* out = static_cast<OUT*>(p.out);
        uint32_t n = 0;
        const uint32_t acc_empty_at = CG == 2 ? map_to(acc_empty0, 0) : acc_empty0;
        pdl_wait();
        for (uint32_t tile = first; tile < p.tiles; tile += step) {
            const uint32_t tv = tile / p.tiles_t, tt = tile - tv * p.tiles_t, t0 = tt * p.tile_t;
            const uint32_t v = (tv * CG + rank) * kTileV + quad * 32 + lane;
            const uint32_t rows = min(p.tile_t, p.T - t0);
            const float sw = p.w_scale && v < p.V ? p.w_scale[v] : 1.f;
            float sum[kMaxBlocks][32];
            const uint32_t acc = acc_of(n);
            if (!mbar_wait_warp(acc_full0 + 8 * acc, acc_phase(n), s_abort)) break;
            ++n;
            fence_after();
#pragma unroll
            for (uint32_t i = 0; i < kMaxBlocks; ++i) {
                const uint32_t c0 = (share + kShares * i) * 32;
                if (c0 < rows) tmem_load32(tmem + ((quad * 32) << 16) + acc * (kMaxTileT / 2) + c0, sum[i]);
            }
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) mbar_arrive_at(acc_empty_at + 8 * acc);
                else mbar_arrive(acc_empty0 + 8 * acc);
            }
#pragma unroll
            for (uint32_t i = 0; i < kMaxBlocks; ++i) {
                const uint32_t c0 = (share + kShares * i) * 32;
                if (c0 >= rows) continue;
                const float row_scale = p.x_scale && c0 + lane < rows ? p.x_scale[t0 + c0 + lane] : 1.f;
                OUT* o = out + (uint64_t)(t0 + c0) * p.out_stride + v;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float y = sum[i][c] * sw * __shfl_sync(0xFFFFFFFFu, row_scale, c);
                    if (v < p.V && c0 + c < rows) *o = from_f32<OUT>(y);
                    o += p.out_stride;
                }
            }
        }
    }
    // Everything issued is finished before shared memory and TMEM go; after an abort the copies
    // and products in flight end by themselves, and these waits are bounded like the others.
    if (warp == kMmaWarp && lane == 0) {  // (in both CTAs of a pair: the commit arrives in both)
        uint32_t dummy = 0;
        (void)mbar_wait(drain, 0, &dummy);
    }
    if (lane == 0 && *s_abort) {
        uint32_t dummy = 0;
        if (rank == 0)  // (the even CTA's barriers count the pair's copies)
            for (uint32_t i = issued < p.stages ? 0 : issued - p.stages; i < issued; ++i)
                (void)mbar_wait(full0 + 8 * (i % p.stages), (i / p.stages) & 1, &dummy);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();  // neither CTA leaves while the other may write to it
    fence_after();
    if (warp == kMmaWarp) {
        if constexpr (CG == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kColumns));
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kColumns));
    }
    if (threadIdx.x == 0 && *s_abort) flag(p.status, LP_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ host

// Map of a matrix of bytes [rows][cols], in boxes of 128 bytes, swizzled, by box_rows rows.
bool encode_codes(CUtensorMap* map, const void* ptr, uint64_t rows, uint64_t cols, uint64_t stride, uint32_t box_rows) {
    const EncodeFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {stride};
    const cuuint32_t box[2] = {kSliceBytes, box_rows}, step[2] = {1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Map of `tiles` tiles of scales of 512 bytes, in boxes of box_tiles.
bool encode_scales(CUtensorMap* map, const void* ptr, uint64_t tiles, uint32_t box_tiles) {
    const EncodeFn f = encode_fn();
    if (!f) return false;
    const cuuint64_t dims[2] = {128, tiles}, strides[1] = {512};
    const cuuint32_t box[2] = {128, box_tiles}, step[2] = {1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(ptr), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Project4Launch {
    CUtensorMap w, x, ws, xs;
    Project4Params p;
    size_t smem;
    unsigned grid;
};

template <int BLOCK, typename OUT, int CG>
lp_status launch_project4(const Project4Launch& l, lp_stream_t stream) {
    static std::atomic<uint64_t> smem_set;
    auto kernel = k_project4<BLOCK, OUT, CG>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), kSmemBudget, &smem_set)) return LP_ERR_CUDA;
    return launch(kernel, dim3(l.grid), kThreads, l.smem, stream, CG, l.w, l.x, l.ws, l.xs, l.p);
}
template <int BLOCK, int CG>
lp_status launch_project4(const Project4Launch& l, uint32_t out_dtype, lp_stream_t s) {
    if (out_dtype == LP_F32) return launch_project4<BLOCK, float, CG>(l, s);
    if (out_dtype == LP_BF16) return launch_project4<BLOCK, __nv_bfloat16, CG>(l, s);
    return launch_project4<BLOCK, __half, CG>(l, s);
}

}  // namespace

extern "C" lp_status lp_head_project4(const void* x, uint64_t x_stride, const void* x_scales, const float* x_row_scale,
                                      uint32_t T, uint32_t H, uint32_t block, const void* weight, uint64_t weight_stride,
                                      const void* weight_scales, const float* weight_row_scale, uint32_t V, void* out,
                                      uint32_t out_dtype, uint64_t out_stride, void* workspace, size_t workspace_bytes,
                                      lp_stream_t stream) {
    if (T == 0 || V == 0 || H == 0) return LP_ERR_SHAPE;
    if (!x || !x_scales || !weight || !weight_scales || !out) return LP_ERR_NULL;
    if (out_dtype != LP_F32 && out_dtype != LP_BF16 && out_dtype != LP_F16) return LP_ERR_DTYPE;
    if ((block != 16 && block != 32) || H % 32 || T > 0x7FFFFF00u || V > 0x7FFFFF00u || H > 0x7FFFFF00u) return LP_ERR_SHAPE;
    if (x_stride < H / 2 || weight_stride < H / 2 || x_stride % 16 || weight_stride % 16 || out_stride < V) return LP_ERR_SHAPE;
    if (!aligned_to(x, 16) || !aligned_to(weight, 16) || !aligned_to(x_scales, 16) || !aligned_to(weight_scales, 16) ||
        !aligned_to(x_row_scale, 4) || !aligned_to(weight_row_scale, 4) || !aligned_to(out, dtype_bytes(out_dtype)))
        return LP_ERR_SHAPE;
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < kHeaderBytes) return LP_ERR_WORKSPACE;
    Project4Launch l = {};
    Project4Params& p = l.p;
    p.col_tiles = ((H + block - 1) / block + 3) / 4;
    const uint64_t w_tiles = (uint64_t)((V + 127) / 128) * p.col_tiles, x_tiles = (uint64_t)((T + 127) / 128) * p.col_tiles;
    if (w_tiles > 0x7FFFFFFFu || x_tiles > 0x7FFFFFFFu) return LP_ERR_SHAPE;  // (coordinates of copies)
    const int sms = sm_count();
    if (sms == 0) return LP_ERR_CUDA;
    p.x_scale = x_row_scale;
    p.w_scale = weight_row_scale;
    p.out = out;
    p.status = static_cast<uint32_t*>(workspace);
    p.out_stride = out_stride;
    p.T = T;
    p.V = V;
    p.H = H;
    p.slices = (H + kSlice - 1) / kSlice;
    const uint32_t cg = T > 128 ? 2 : 1, unit = 16 * cg;
    p.tile_t = T > kMaxTileT ? kMaxTileT : (T + unit - 1) / unit * unit;  // (several tiles: whole blocks of 128 rows)
    p.tiles_t = (T + p.tile_t - 1) / p.tile_t;
    const uint64_t tiles = (uint64_t)((V + cg * kTileV - 1) / (cg * kTileV)) * p.tiles_t;
    if (tiles > 0x7FFFFFFFu) return LP_ERR_SHAPE;
    p.tiles = (uint32_t)tiles;
    p.acc_shift = p.tile_t <= kMaxTileT / 2;
    const uint32_t scale_bytes = kSlice / block * 128, columns = scale_bytes / 128 * (1 + cg);
    const uint32_t stage_bytes = kStageW + p.tile_t / cg * kSliceBytes + (1 + cg) * scale_bytes;
    p.stages = (kSmemBudget - kControlBytes) / stage_bytes;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    if (p.stages > (kColumns - kScaleColumns) / columns) p.stages = (kColumns - kScaleColumns) / columns;
    l.smem = kControlBytes + p.stages * stage_bytes;
    // instruction: e2m1 operands, K-major, M = 128 lanes a CTA; the scales' type: 1 for e8m0
    p.idesc = (1u << 7) | (1u << 10) | ((block == 32 ? 1u : 0u) << 23) | ((cg * kTileV >> 7) << 27);
    const uint32_t box_tiles = kSlice / (4 * block);
    if (!encode_codes(&l.w, weight, V, H / 2, weight_stride, kTileV) ||
        !encode_codes(&l.x, x, T, H / 2, x_stride, p.tile_t / cg) || !encode_scales(&l.ws, weight_scales, w_tiles, box_tiles) ||
        !encode_scales(&l.xs, x_scales, x_tiles, box_tiles))
        return LP_ERR_CUDA;
    const uint32_t units = (uint32_t)sms / cg;
    l.grid = cg * (p.tiles < units ? p.tiles : units);
    if (block == 16) return cg == 2 ? launch_project4<16, 2>(l, out_dtype, stream) : launch_project4<16, 1>(l, out_dtype, stream);
    return cg == 2 ? launch_project4<32, 2>(l, out_dtype, stream) : launch_project4<32, 1>(l, out_dtype, stream);
}
