// Projection of hidden states to logits with low-rank adapters (include/lp_head.h):
//     out[t, v] = sx[t] sw[v] sum_h x[t, h] W[v, h] + sum_j u[t, j] B_a[v, j],
//     u[t, j]   = s_a sx[t] sum_h x[t, h] A_a[j, h],   a = adapter of row t's request.
//
// The product runs on the tensor cores with the vocabulary on the accumulator's lanes: a
// tile is 128 vocabulary rows (256 of a pair of CTAs) by N rows of x (at most 256), so that a
// decode step reads W once and pads little, and a warp's 32 lanes hold 32 neighbouring logits of
// one output row (coalesced stores without a transpose). One thread issues TMA copies of
// 128-byte-wide slices of W and x into a ring of stages, one issues tcgen05.mma from them into
// one of two to eight accumulators in TMEM (what 512 columns hold), and twelve warps empty the
// others meanwhile. Kernels are persistent; consecutive tiles share their W rows.
//
// u is computed first, by its own small kernel (lp_adapters.cu); the product starts while that
// still runs and waits for it only at the end of its first tile. Where 32 rows of a tile have
// one adapter or two, u B_a^T is a product on the tensor cores as well, with u as three 16-bit
// parts (24 bits, what f32 has); other rows, and tiles of single CTAs, are multiplied by the
// epilogue in f32, adapter by adapter, with tiles of B_a copied ahead of it.
//
// Bound by HBM (W) up to about 128 rows, by the tensor cores above. Measured, us (W at HBM's
// measured rate, or the products at a large library product's): one row, V = 128256, H = 4096
// bf16 162 (155); 256 rows 183 (155); 2048 rows, V = 32000 bf16 286 and f32 327 (287); e4m3 48
// rows of V = 152064 with 12 adapters of rank 32 127-130 (114).
#include "lp_adapters.h"
#include "lp_tcgen05.h"

namespace {

using namespace lph;

constexpr uint32_t kTileV = 128;                  // vocabulary rows of a CTA's tile (accumulator lanes)
constexpr uint32_t kSliceBytes = 128;             // bytes of the contracted dimension per stage
constexpr uint32_t kStageW = kTileV * kSliceBytes;
constexpr uint32_t kMaxStages = 12;
constexpr uint32_t kEpilogueWarps = 12;
constexpr uint32_t kShares = kEpilogueWarps / 4;  // epilogue warps of one quadrant of lanes
constexpr uint32_t kMaxDepth = 3;                 // buffers a share has for tiles of the adapters' B
constexpr uint32_t kMaxSlots = kShares * kMaxDepth;
// Warps: the epilogue's (warp % 4 is the quadrant of lanes a warp may read), then one that
// issues copies, one that issues products, one that fills the adapters' buffers.
constexpr uint32_t kCopyWarp = kEpilogueWarps, kMmaWarp = kEpilogueWarps + 1, kBufferWarp = kEpilogueWarps + 2;
constexpr uint32_t kThreads = (kEpilogueWarps + 3) * 32;
constexpr uint32_t kControlBytes = 1024 + 512;    // barriers and words, and the alignment of the ring
// Slices summed in the tensor core before an f32 addition: f32 logits of 16-bit inputs. Half as
// many for tiles of few rows, which wait for HBM (64 rows on V = 128256, H = 4096: 180.9 us both
// ways, and half the error; with 256 rows 207.5 against 199.3).
constexpr uint32_t kPromoteSlices = 8, kPromoteFewRows = 64;

struct ProjectParams {
    const float* x_scale;
    const float* w_scale;
    const void* lora_b;            // [A][V][rank]
    const float* u;                // [T][u_cols]
    const float* factor;           // [T]
    const unsigned char* groups;   // [tiles_t] TileGroups, kGroupBytes apart
    void* out;
    uint32_t* status;
    uint64_t out_stride;
    uint32_t T, V, rank;
    uint32_t u_cols;               // rank rounded up to 16
    uint32_t b_cols;               // columns of a B buffer: 16, 32 or 64
    uint32_t depth;                // B buffers of a share
    uint32_t u_smem;               // a tile's u is staged in shared memory (else read from global)
    uint32_t part_stride;          // rows of u's parts
    uint32_t tile_t;               // N
    uint32_t tiles_t, tiles, slices, stages;
    uint32_t chunk;                // slices summed in one accumulator pass
    uint32_t acc_cols;             // TMEM columns of one accumulator
    uint32_t acc_shift;            // log2 of the number of accumulators
    uint32_t idesc, lora_idesc;    // instruction descriptors: of x W^T, of the adapters' part
    uint32_t tensor;               // blocks of rows with one adapter run on the tensor cores
    uint32_t apart;                // all with an accumulator of their own: their sum has another
                                   // scale (e4m3) or a factor a row (f16)
    uint64_t lora_bytes;           // of lora_b
    uint32_t lora_f16;             // lora_b is f16 (else bf16)
    uint32_t lora_tma;             // lora_b's rows are whole 16-byte pieces (swizzled tiles in the buffers)
    uint32_t early;                // the inputs are complete when this kernel starts (u may not be)
};

constexpr uint32_t kMaxAccs = 8;
constexpr uint32_t kBarriers = 2 * kMaxStages + 2 * kMaxSlots + 2 * kMaxAccs + 2;

template <bool FP8, int CG>
__device__ __forceinline__ void mma(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
#define LPH_MMA(GROUP, KIND)                                                                       \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"                               \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem), \
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory")
    if constexpr (FP8 && CG == 2) LPH_MMA("2", "f8f6f4");
    else if constexpr (FP8) LPH_MMA("1", "f8f6f4");
    else if constexpr (CG == 2) LPH_MMA("2", "f16");
    else LPH_MMA("1", "f16");
#undef LPH_MMA
}

__device__ __forceinline__ void tmem_store32(uint32_t addr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};"
        ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
          "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
          "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
          "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31]), "r"(addr) : "memory");
}

// Eight columns of the accumulator, one by one.
__device__ __forceinline__ void tmem_load_columns(uint32_t base, const uint32_t (&col)[8], float (&v)[8]) {
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[i]) : "r"(base + col[i]) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 ::"memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Two f32 at a time: a * b + c.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t pair(float2 f) {
    return (uint64_t)__float_as_uint(f.x) | ((uint64_t)__float_as_uint(f.y) << 32);
}

// Byte offset of 16-byte piece `piece` of row `row` in a B buffer of `cols` columns: rows of
// 32, 64 or 128 bytes, the pieces swizzled as TMA writes them, so that the 32 rows that a
// warp reads spread over the banks.
__device__ __forceinline__ uint32_t b_offset(uint32_t row, uint32_t piece, uint32_t cols) {
    const uint32_t off = row * cols * 2 + piece * 16;
    return off ^ ((off >> 3) & (cols * 2 - 16));
}

// Where the chunk that begins at slice k0 ends. A tile's first is half as long again: the
// epilogue is still storing the tile before, from the other accumulator.
__device__ __forceinline__ uint32_t chunk_end(const ProjectParams& p, uint32_t k0) {
    return k0 + min(p.slices - k0, k0 ? p.chunk : p.chunk + p.chunk / 2);
}
__device__ __forceinline__ const TileGroups* tile_groups(const ProjectParams& p, uint32_t tt) {
    return reinterpret_cast<const TileGroups*>(p.groups + (size_t)tt * kGroupBytes);
}
// Lines of u's parts that a stage holds for a run of `blocks` blocks beside B_a: all that it has,
// where the rows of x in a stage leave the room (a short run has little to compute, and with a
// stage a line the copies of the product's next slices started too late for it: 2048 x 32000
// with ragged adapters of rank 64: 441 us so, 436 with all in one), or one.
__device__ __forceinline__ uint32_t lines_a_stage(uint32_t lines, uint32_t blocks, uint32_t N) {
    return lines * blocks * kBlock <= N ? lines : 1;
}
// A tile's runs: the count and the first four are fetched when the tile begins, long before
// they are used.
struct RunList {
    const TileGroups* g;
    uint32_t runs;
    uint2 head[4];
    __device__ __forceinline__ void fetch(const TileGroups* groups) {
        g = groups;
        runs = g->runs;
#pragma unroll
        for (int i = 0; i < 4; ++i) head[i] = g->run[i];
    }
    __device__ __forceinline__ uint2 at(uint32_t r) const {
        return r == 0 ? head[0] : r == 1 ? head[1] : r == 2 ? head[2] : r == 3 ? head[3] : g->run[r];
    }
};

// PROMOTE: f32 logits of 16-bit inputs. The tensor core's f32 accumulator drops the bits
// below its last place at every step, always towards zero: over a contraction of 4096 that
// adds up to 4.4e-6 of the result, against 6e-7 of rounded f32 sums. So the accumulator is
// emptied into registers every 8 slices (512 products; 4 for tiles of few rows; the first time
// after half as many again), and those are summed with rounding: 4.8e-7 (4 slices 2.5e-7, 2
// 1.6e-7, 16 1.0e-6).
// It costs 2048 rows on V = 32000 327 us instead of 286. Rounded outputs (16 bits) and e4m3
// products (few bits) do not need it.
template <bool FP8, typename OUT, int CG, bool PROMOTE, bool LORA>
__global__ void __launch_bounds__(kThreads, 1)
k_project(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
          const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_lora_b,
          const __grid_constant__ CUtensorMap map_parts, const ProjectParams p) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* ring = smem_raw + (base - smem_u32(smem_raw));
    const uint32_t N = p.tile_t, stage_bytes = kStageW + N / CG * kSliceBytes;
    const uint32_t uc = p.u_cols, slot_bytes = kTileV * p.b_cols * 2;
    unsigned char* s_b = ring + p.stages * stage_bytes;                         // [shares][depth][128][b_cols]
    float* s_u = reinterpret_cast<float*>(s_b + kShares * p.depth * slot_bytes);  // [N][uc]
    float* s_scale = s_u + (LORA && p.u_smem ? N * uc : 0);                     // [N]
    TileGroups* s_groups = reinterpret_cast<TileGroups*>(s_scale + (FP8 && LORA ? N : 0));
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<unsigned char*>(s_groups) +
                                                 (LORA ? sizeof(TileGroups) : 0));
    volatile uint32_t* s_abort = reinterpret_cast<uint32_t*>(bars + kBarriers);
    uint32_t* s_tmem = const_cast<uint32_t*>(s_abort) + 1;
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * kMaxStages, b_full0 = empty0 + 8 * kMaxStages,
                   b_empty0 = b_full0 + 8 * kMaxSlots, acc_full0 = b_empty0 + 8 * kMaxSlots,
                   acc_empty0 = acc_full0 + 8 * kMaxAccs, drain = acc_empty0 + 8 * kMaxAccs, staging = drain + 8;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank = 0;
    if constexpr (CG == 2) asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const uint32_t first = blockIdx.x / CG, step = gridDim.x / CG;  // tiles of this CTA (pair)
    // the n-th filling: its accumulator, and the phase of that one's barriers
    const auto acc_of = [&](uint32_t n) { return n & ((1u << p.acc_shift) - 1); };
    const auto acc_phase = [&](uint32_t n) { return n >> p.acc_shift & 1; };

    pdl_trigger();
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < p.stages; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (uint32_t i = 0; LORA && i < kShares * p.depth; ++i) {
            mbar_init(b_full0 + 8 * i, 1);
            mbar_init(b_empty0 + 8 * i, 4);  // the share's warps
        }
        for (uint32_t i = 0; i < 1u << p.acc_shift; ++i) {
            mbar_init(acc_full0 + 8 * i, 1);
            mbar_init(acc_empty0 + 8 * i, kEpilogueWarps * CG);
        }
        mbar_init(drain, 1);
        mbar_init(staging, kEpilogueWarps);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        if constexpr (CG == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                         "r"(p.acc_cols << p.acc_shift) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(s_tmem)),
                         "r"(p.acc_cols << p.acc_shift) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();  // the other CTA's barriers are ready too
    fence_after();
    const uint32_t tmem = *s_tmem;

    uint32_t issued = 0;    // stages the producer has started copies into
    if (warp == kCopyWarp) {
        if (lane == 0) {
            if (!p.early) pdl_wait();
            uint64_t once, keep;  // W is read once per row of tiles, x by every tile
            asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
            asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
            const uint64_t w_policy = p.tiles_t == 1 ? once : keep;
            const uint32_t slice_elems = FP8 ? kSliceBytes : kSliceBytes / 2;
            uint32_t s = 0, phase = 0;
            bool ok = true;
            for (uint32_t tile = first; ok && tile < p.tiles; tile += step) {
                const uint32_t tv = tile / p.tiles_t, tt = tile - tv * p.tiles_t;
                const int v0 = (int)((tv * CG + rank) * kTileV), t0 = (int)(tt * N + rank * (N / CG));
                RunList list;
                if (LORA && CG == 2 && p.tensor && tile != first) list.fetch(tile_groups(p, tt));
                for (uint32_t k = 0;; ++k) {
                    if constexpr (LORA && CG == 2) {
                        if (p.tensor && k == p.slices) {
                            if (tile == first) {
                                pdl_wait();
                                list.fetch(tile_groups(p, tt));
                            }
                            // runs of blocks with one adapter: B_a in W's place, the parts of u in x's
                            for (uint32_t r = 0; ok && r < list.runs; ++r) {
                                const uint2 run = list.at(r);
                                const uint32_t a = run.y, b0 = run.x >> 8 & 0xFF, n = run.x & 0xFF;
                                constexpr uint32_t kHalf = kBlock / CG;  // rows of a block that a CTA holds
                                const uint32_t lines = part_rows(p.rank), group = lines_a_stage(lines, n, N);
                                for (uint32_t l0 = 0; l0 < lines; l0 += group) {
                                    if (!mbar_wait(empty0 + 8 * s, phase ^ 1, s_abort)) { ok = false; break; }
                                    const uint32_t dst = base + s * stage_bytes, bar = map_to(full0 + 8 * s, 0);
                                    if (rank == 0) mbar_expect(full0 + 8 * s, CG * (kStageW + group * n * kHalf * kSliceBytes));
                                    tma_2d<CG>(dst, &map_lora_b, 0, (int)(a * p.V) + v0, bar, keep);
                                    for (uint32_t i = 0; i < group * n; ++i) {
                                        const uint32_t line = l0 + i / n, block = i % n;
                                        tma_2d<CG>(dst + kStageW + i * kHalf * kSliceBytes, &map_parts, 0,
                                                   (int)(line * p.part_stride + tt * N + b0 * kBlock + (rank * n + block) * kHalf),
                                                   bar, keep);
                                    }
                                    ++issued;
                                    if (++s == p.stages) { s = 0; phase ^= 1; }
                                }
                            }
                        }
                    }
                    if (!ok || k == p.slices) break;
                    if (!mbar_wait(empty0 + 8 * s, phase ^ 1, s_abort)) { ok = false; break; }
                    const uint32_t dst = base + s * stage_bytes;
                    const uint32_t bar = CG == 2 ? map_to(full0 + 8 * s, 0) : full0 + 8 * s;
                    if (rank == 0) mbar_expect(full0 + 8 * s, CG * stage_bytes);
                    tma_2d<CG>(dst, &map_w, (int)(k * slice_elems), v0, bar, w_policy);
                    tma_2d<CG>(dst + kStageW, &map_x, (int)(k * slice_elems), t0, bar, keep);
                    ++issued;
                    if (++s == p.stages) { s = 0; phase ^= 1; }
                }
            }
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0 && rank == 0) {
            // (nothing to wait for before the copies begin; the bounded waits below are for this
            // kernel's own work, not for an earlier one that let this one launch early)
            if (!p.early) pdl_wait();
            uint32_t s = 0, phase = 0, n = 0;
            bool ok = true;
            for (uint32_t tile = first; ok && tile < p.tiles; tile += step) {
                RunList list;
                if (LORA && CG == 2 && p.tensor && tile != first) list.fetch(tile_groups(p, tile % p.tiles_t));
                for (uint32_t k0 = 0, k1; ok; k0 = k1) {
                    if constexpr (LORA && CG == 2) {
                        if (p.tensor && k0 == p.slices) {
                            // The adapters' passes: pass 0 into the open accumulator, 1 into the next.
                            if (tile == first) {
                                pdl_wait();
                                list.fetch(tile_groups(p, tile % p.tiles_t));
                            }
                            uint32_t pass = 0;
                            bool open = !p.apart;  // the product's own accumulator
                            for (uint32_t r = 0; ok && r < list.runs; ++r) {
                                const uint2 run = list.at(r);
                                const uint32_t to = run.x >> 24, blocks = run.x & 0xFF;
                                if ((run.x >> 16 & 0xFF) != pass) {
                                    if (open) {
                                        mma_commit<CG>(acc_full0 + 8 * acc_of(n));
                                        ++n;
                                    }
                                    pass = 1;
                                    open = mbar_wait(acc_empty0 + 8 * acc_of(n), acc_phase(n) ^ 1, s_abort);
                                    if (!open) { ok = false; break; }
                                }
                                const uint32_t idesc = p.lora_idesc | ((blocks * kBlock >> 3) << 17);
                                const uint32_t lines = part_rows(p.rank), group = lines_a_stage(lines, blocks, N);
                                for (uint32_t l0 = 0; l0 < lines; l0 += group) {
                                    if (!mbar_wait(full0 + 8 * s, phase, s_abort)) { ok = false; break; }
                                    fence_after();
                                    const uint64_t a = matrix_desc(base + s * stage_bytes);
                                    for (uint32_t line = l0; line < l0 + group; ++line) {
                                        const uint64_t b = matrix_desc(base + s * stage_bytes + kStageW +
                                                                       (line - l0) * blocks * (kBlock / CG) * kSliceBytes);
                                        // 16 columns of the parts a step; B_a's start again with each part
                                        for (uint32_t i = 0; i < 4; ++i) {
                                            const uint32_t column = line * 64 + i * 16, part = column / p.b_cols,
                                                           j = column - part * p.b_cols;
                                            if (part < 3 && j < uc)
                                                mma<false, CG>(tmem + acc_of(n) * p.acc_cols + to * kBlock, a + j / 8, b + 2 * i,
                                                               idesc, pass ? (line | i) : 1u);
                                        }
                                    }
                                    mma_commit<CG>(empty0 + 8 * s);
                                    if (++s == p.stages) { s = 0; phase ^= 1; }
                                }
                            }
                            if (!ok) break;
                            if (open) {
                                mma_commit<CG>(acc_full0 + 8 * acc_of(n));
                                ++n;
                            }
                        }
                    }
                    if (k0 >= p.slices) break;
                    const uint32_t acc = acc_of(n);
                    k1 = chunk_end(p, k0);
                    if (!mbar_wait(acc_empty0 + 8 * acc, acc_phase(n) ^ 1, s_abort)) { ok = false; break; }
                    fence_after();
                    for (uint32_t k = k0; k < k1; ++k) {
                        if (!mbar_wait(full0 + 8 * s, phase, s_abort)) { ok = false; break; }
                        fence_after();
                        const uint64_t a = matrix_desc(base + s * stage_bytes);
                        const uint64_t b = matrix_desc(base + s * stage_bytes + kStageW);
#pragma unroll
                        for (uint32_t i = 0; i < kSliceBytes / 32; ++i)  // 32 bytes of the contracted dimension each
                            mma<FP8, CG>(tmem + acc * p.acc_cols, a + 2 * i, b + 2 * i, p.idesc, (k - k0) | i);
                        mma_commit<CG>(empty0 + 8 * s);
                        if (++s == p.stages) { s = 0; phase ^= 1; }
                    }
                    if (!ok) break;
                    if (LORA && CG == 2 && p.tensor && !p.apart && k1 == p.slices) continue;  // pass 0 continues it
                    mma_commit<CG>(acc_full0 + 8 * acc);
                    ++n;
                }
            }
            mma_commit<CG>(drain);  // arrives once every product issued above has finished
        }
    } else if (warp == kBufferWarp) {
        // Tiles of the adapters' B, in the order the epilogue takes them.
        if constexpr (LORA) {
            pdl_wait();
            uint64_t once;
            asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
            uint32_t used[kShares] = {};  // buffers of each share filled so far
            bool ok = true;
            for (uint32_t tile = first; ok && tile < p.tiles; tile += step) {
                const uint32_t tv = tile / p.tiles_t, tt = tile - tv * p.tiles_t;
                const uint32_t v0 = (tv * CG + rank) * kTileV;
                const TileGroups* g = tile_groups(p, tt);
                const uint32_t items = v0 < p.V ? g->items : 0u;
                for (uint32_t k = 0; k < items; ++k) {
                    const uint32_t a = g->item[k], share = k % kShares;
                    if (a == kNoAdapter) break;
                    uint32_t count = 0;
#pragma unroll
                    for (uint32_t i = 0; i < kShares; ++i) count = i == share ? used[i]++ : count;
                    const uint32_t s = share * p.depth + count % p.depth, phase = count / p.depth & 1;
                    if (!mbar_wait_warp(b_empty0 + 8 * s, phase ^ 1, s_abort)) { ok = false; break; }
                    const uint32_t bar = b_full0 + 8 * s;
                    if (p.lora_tma) {
                        if (lane == 0) {
                            mbar_expect(bar, slot_bytes);
                            tma_2d<1>(smem_u32(s_b) + s * slot_bytes, &map_b, 0, (int)(a * p.V + v0), bar, once);
                        }
                        __syncwarp();
                    } else {
                        // Rows of any length are one stretch of memory: copied as it is, from the
                        // 16-byte boundary before it to the one after it, or to the last one within
                        // the tensor, whose last bytes are then copied one value at a time.
                        const uint64_t begin = ((uint64_t)a * p.V + v0) * p.rank * 2, from = begin & ~15ull;
                        const uint64_t end = begin + (uint64_t)min(kTileV, p.V - v0) * p.rank * 2;
                        const uint64_t limit = p.lora_bytes & ~15ull;
                        const uint64_t upto = (end + 15) & ~15ull;
                        const uint32_t bytes = (uint32_t)((upto < limit ? upto : limit) - from);
                        unsigned char* dst = s_b + s * slot_bytes;
                        if (from + bytes + 2 * lane < end)
                            *reinterpret_cast<uint16_t*>(dst + bytes + 2 * lane) = *reinterpret_cast<const uint16_t*>(
                                static_cast<const unsigned char*>(p.lora_b) + from + bytes + 2 * lane);
                        __syncwarp();
                        if (lane == 0) {
                            mbar_expect(bar, bytes);
                            if (bytes)
                                bulk_copy(smem_u32(dst), static_cast<const unsigned char*>(p.lora_b) + from, bytes, bar);
                        }
                        __syncwarp();
                    }
                }
            }
            // (every copy started ends, whether or not its tile is still taken)
            if (*s_abort) {
                uint32_t dummy = 0;
                for (uint32_t i = 0; i < kShares; ++i)
                    for (uint32_t c = used[i] < p.depth ? 0 : used[i] - p.depth; c < used[i]; ++c)
                        (void)mbar_wait_warp(b_full0 + 8 * (i * p.depth + c % p.depth), c / p.depth & 1, &dummy);
            }
        }
    } else {
        // The quadrant of lanes this warp may read, and its share of the columns: the blocks
        // of 32 whose number is `share` modulo kShares.
        const uint32_t quad = warp & 3, share = warp >> 2;
        const uint32_t et = threadIdx.x;
        OUT* out = static_cast<OUT*>(p.out);
        uint32_t n = 0, staged = 0xFFFFFFFFu, staging_phase = 0, used = 0;
        const uint32_t acc_empty_at = CG == 2 ? map_to(acc_empty0, 0) : acc_empty0;
        // all epilogue warps have come here (a bounded wait, as everywhere: no warp can be
        // left behind by one that gave up)
        const auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(staging);
            const bool ok = mbar_wait_warp(staging, staging_phase, s_abort);
            staging_phase ^= 1;
            return ok;
        };
        const auto release = [&](uint32_t acc) {
            fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) mbar_arrive_at(acc_empty_at + 8 * acc);
                else mbar_arrive(acc_empty0 + 8 * acc);
            }
        };
        pdl_wait();
        for (uint32_t tile = first; tile < p.tiles; tile += step) {
            const uint32_t tv = tile / p.tiles_t, tt = tile - tv * p.tiles_t, t0 = tt * N;
            const uint32_t v0 = (tv * CG + rank) * kTileV, v = v0 + quad * 32 + lane;
            const uint32_t rows = min(N, p.T - t0);
            [[maybe_unused]] const TileGroups* g = LORA ? tile_groups(p, tt) : nullptr;
            if constexpr (LORA) {
                const uint32_t items = g->items;
                if (items && tt != staged) {  // the lists, u and scales in shared memory
                    if (!meet()) break;
                    const uint4* words = reinterpret_cast<const uint4*>(g);
                    for (uint32_t i = et; i < sizeof(TileGroups) / 16; i += kEpilogueWarps * 32)
                        reinterpret_cast<uint4*>(s_groups)[i] = words[i];
                    if (p.u_smem) {
                        const float4* src = reinterpret_cast<const float4*>(p.u + (uint64_t)t0 * uc);
                        for (uint32_t i = et; i < rows * uc / 4; i += kEpilogueWarps * 32)
                            reinterpret_cast<float4*>(s_u)[i] = src[i];
                    }
                    if constexpr (FP8)
                        for (uint32_t i = et; i < rows; i += kEpilogueWarps * 32) s_scale[i] = p.x_scale[t0 + i];
                    if (!meet()) break;
                    staged = tt;
                }
            }
            // of row c of a block, from the lane that holds it
            const auto of_row = [&](const float* per_row, uint32_t c0) {
                return c0 + lane < rows ? per_row[t0 + c0 + lane] : 0.f;
            };
            const float sw = FP8 && v < p.V ? p.w_scale[v] : 1.f;
            uint32_t acc = acc_of(n);
            const uint32_t lanes = (quad * 32) << 16;
            if constexpr (PROMOTE) {
                float sum[(kMaxTileT / 32 + kShares - 1) / kShares][32];
                bool ok = true;
#pragma unroll
                for (uint32_t i = 0; i < (kMaxTileT / 32 + kShares - 1) / kShares; ++i)
#pragma unroll
                    for (int c = 0; c < 32; ++c) sum[i][c] = 0.f;
                for (uint32_t k0 = 0;;) {
                    acc = acc_of(n);
                    if (!mbar_wait_warp(acc_full0 + 8 * acc, acc_phase(n), s_abort)) { ok = false; break; }
                    ++n;
                    fence_after();
                    k0 = chunk_end(p, k0);
#pragma unroll
                    for (uint32_t i = 0; i < (kMaxTileT / 32 + kShares - 1) / kShares; ++i) {
                        const uint32_t c0 = (share + kShares * i) * 32;
                        if (c0 >= N) continue;
                        const uint32_t at = tmem + lanes + acc * p.acc_cols + c0;
#pragma unroll
                        for (int q = 0; q < 32; q += 16) {
                            float y[16];
                            tmem_load16(at + q, y);
#pragma unroll
                            for (int c = 0; c < 16; ++c) sum[i][q + c] += y[c];
                        }
                    }
                    if (k0 == p.slices) break;
                    release(acc);
                }
                if (!ok) break;
                const uint32_t blocks = LORA && CG == 2 && p.tensor ? g->blocks : 0u;
                if (blocks) {  // pass 1
                    release(acc);
                    acc = acc_of(n);
                    if (!mbar_wait_warp(acc_full0 + 8 * acc, acc_phase(n), s_abort)) break;
                    ++n;
                    fence_after();
                    const uint32_t columns = tmem + lanes + acc * p.acc_cols;
#pragma unroll
                    for (uint32_t i = 0; i < (kMaxTileT / 32 + kShares - 1) / kShares; ++i) {
                        const uint32_t b = share + kShares * i, c0 = b * 32;
                        if (c0 >= N || !(blocks >> b & 1)) continue;
                        const float factor = p.lora_f16 ? of_row(p.factor, c0) : 1.f;
                        const uint32_t adapters = 1 + (g->second >> b & 1);
                        for (uint32_t k = 0; k < adapters; ++k) {
                            const uint32_t take = g->rows[k][b], from = k ? (g->place >> 4 * b & 15) * 32 : c0;
#pragma unroll
                            for (int q = 0; q < 32; q += 16) {
                                float y[16];
                                tmem_load16(columns + from + q, y);
                                if (p.lora_f16) {
#pragma unroll
                                    for (int c = 0; c < 16; ++c) y[c] *= __shfl_sync(0xFFFFFFFFu, factor, q + c);
                                }
#pragma unroll
                                for (int c = 0; c < 16; ++c) sum[i][q + c] += take >> (q + c) & 1 ? y[c] : 0.f;
                            }
                        }
                    }
                    // (a block's columns may hold another's second sums)
                    fence_before();
                    if (!meet()) break;
                    fence_after();
                }
#pragma unroll
                for (uint32_t i = 0; i < (kMaxTileT / 32 + kShares - 1) / kShares; ++i) {
                    const uint32_t c0 = (share + kShares * i) * 32;
                    if (c0 < N) tmem_store32(tmem + lanes + acc * p.acc_cols + c0, sum[i]);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            } else {
                if (!mbar_wait_warp(acc_full0 + 8 * acc, acc_phase(n), s_abort)) break;
                fence_after();
                ++n;
            }
            const uint32_t listed = LORA ? g->listed : 0u, items = LORA ? g->items : 0u;
            const uint32_t blocks = LORA && CG == 2 && p.tensor ? g->blocks : 0u;
            if constexpr (LORA && CG == 2 && !PROMOTE) {
                // With pass 1 the result moves to that pass's accumulator, so that the product's
                // is free for the next tile's before the stores begin.
                if (blocks) {
                    const uint32_t from = tmem + lanes + acc * p.acc_cols;
                    const uint32_t main = acc, second = g->second;
                    acc = acc_of(n);
                    if (!mbar_wait_warp(acc_full0 + 8 * acc, acc_phase(n), s_abort)) break;
                    fence_after();
                    ++n;
                    const uint32_t to = tmem + lanes + acc * p.acc_cols;
                    // the product of block b in y, e4m3's with its scales
                    const auto load_product = [&](uint32_t b, bool scaled, float (&y)[32]) {
                        tmem_load32(from + b * 32, y);
                        if (FP8 && scaled) {
                            const float row_scale = of_row(p.x_scale, b * 32);
#pragma unroll
                            for (int c = 0; c < 32; ++c) y[c] *= sw * __shfl_sync(0xFFFFFFFFu, row_scale, c);
                        }
                    };
                    // and block b's sums at block `at` of the pass, of the rows in `take`
                    const auto add_sums = [&](uint32_t b, uint32_t at, uint32_t take, float (&y)[32]) {
                        float z[32];
                        tmem_load32(to + at * 32, z);
                        if (p.lora_f16) {
                            const float factor = of_row(p.factor, b * 32);
#pragma unroll
                            for (int c = 0; c < 32; ++c) z[c] *= __shfl_sync(0xFFFFFFFFu, factor, c);
                        }
#pragma unroll
                        for (int c = 0; c < 32; ++c) y[c] += take >> c & 1 ? z[c] : 0.f;
                    };
                    if (second) {  // those lie where other blocks' results go
                        for (uint32_t b = share; b < N / 32; b += kShares) {
                            if (!(second >> b & 1)) continue;
                            float y[32];
                            load_product(b, true, y);
                            add_sums(b, g->place >> 4 * b & 15, g->rows[1][b], y);
                            tmem_store32(from + b * 32, y);
                        }
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                        fence_before();
                        if (!meet()) break;
                        fence_after();
                    }
                    for (uint32_t b = share; b * 32 < N; b += kShares) {
                        float y[32];
                        load_product(b, (blocks & ~second) >> b & 1, y);
                        if (blocks >> b & 1) add_sums(b, b, g->rows[0][b], y);
                        tmem_store32(to + b * 32, y);
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    release(main);
                }
            }
            const uint32_t columns = tmem + lanes + acc * p.acc_cols;
            if (!LORA || v0 < p.V) {
                for (uint32_t c0 = share * 32; c0 < N; c0 += kShares * 32) {
                    if (listed >> (c0 / kBlock) & 1) continue;
                    float y[32];
                    tmem_load32(columns + c0, y);
                    if constexpr (FP8) {
                        if (!LORA || !(blocks >> (c0 / kBlock) & 1)) {
                            const float row_scale = of_row(p.x_scale, c0);
#pragma unroll
                            for (int c = 0; c < 32; ++c) y[c] *= sw * __shfl_sync(0xFFFFFFFFu, row_scale, c);
                        }
                    }
                    if (v < p.V) {
                        OUT* o = out + (uint64_t)(t0 + c0) * p.out_stride + v;
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            if (c0 + c < rows) *o = from_f32<OUT>(y[c]);
                            o += p.out_stride;
                        }
                    }
                }
            }
            if (LORA && items && v0 < p.V) {
                if (PROMOTE || blocks) {  // an item's columns may have been written by another share
                    fence_before();
                    if (!meet()) break;
                    fence_after();
                }
                // Item by item: the lane's row of B_a from its buffer, the item's rows of u (the
                // same for every lane), eight rows at a time.
                bool ok = true;
                for (uint32_t k = share; k < items; k += kShares) {  // items go round the shares
                    const uint32_t a = s_groups->item[k];
                    const uint32_t slot = share * p.depth + used % p.depth;
                    if (a != kNoAdapter && !mbar_wait_warp(b_full0 + 8 * slot, used / p.depth & 1, s_abort)) { ok = false; break; }
                    const unsigned char* b_tile = s_b + slot * slot_bytes;
                    const uint32_t begin = s_groups->start[k], end = begin + s_groups->size[k];
                    for (uint32_t i = begin; i < end; i += 8) {
                        uint32_t c[8];
                        float y[8];
#pragma unroll
                        for (int r = 0; r < 8; ++r) c[r] = s_groups->order[min(i + r, end - 1)];
                        tmem_load_columns(columns, c, y);
                        if constexpr (FP8) {
#pragma unroll
                            for (int r = 0; r < 8; ++r) y[r] *= sw * s_scale[c[r]];
                        }
                        if (a != kNoAdapter) {
                            uint64_t y2[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                            for (uint32_t j0 = 0; j0 < uc; j0 += 16) {
                                uint64_t b2[8];
                                uint32_t ws[8];
                                if (p.lora_tma) {
#pragma unroll
                                    for (int q = 0; q < 2; ++q) {
                                        const uint4 w = *reinterpret_cast<const uint4*>(
                                            b_tile + b_offset(quad * 32 + lane, j0 / 8 + q, p.b_cols));
                                        ws[4 * q] = w.x;
                                        ws[4 * q + 1] = w.y;
                                        ws[4 * q + 2] = w.z;
                                        ws[4 * q + 3] = w.w;
                                    }
                                } else {
                                    // (the values past the rank are whatever follows: left out)
                                    const uint16_t* row = reinterpret_cast<const uint16_t*>(
                                        b_tile + (((uint64_t)a * p.V + v0) * p.rank * 2 & 15)) + (quad * 32 + lane) * p.rank + j0;
#pragma unroll
                                    for (int e = 0; e < 8; ++e) {
                                        const uint32_t l = j0 + 2 * e < p.rank ? row[2 * e] : 0u,
                                                       h = j0 + 2 * e + 1 < p.rank ? row[2 * e + 1] : 0u;
                                        ws[e] = l | h << 16;
                                    }
                                }
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    b2[e] = pair(p.lora_f16 ? unpack2(ws[e], __half()) : unpack2(ws[e], __nv_bfloat16()));
#pragma unroll
                                for (int r = 0; r < 8; ++r) {
                                    const ulonglong2* u = reinterpret_cast<const ulonglong2*>(
                                        (p.u_smem ? s_u : p.u + (uint64_t)t0 * uc) + c[r] * uc + j0);
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const ulonglong2 u2 = u[e];
                                        y2[r] = fma2(u2.x, b2[2 * e], y2[r]);
                                        y2[r] = fma2(u2.y, b2[2 * e + 1], y2[r]);
                                    }
                                }
                            }
#pragma unroll
                            for (int r = 0; r < 8; ++r)
                                y[r] += __uint_as_float((uint32_t)y2[r]) + __uint_as_float((uint32_t)(y2[r] >> 32));
                        }
#pragma unroll
                        for (int r = 0; r < 8; ++r)
                            if (i + r < end && v < p.V)
                                out[(uint64_t)(t0 + c[r]) * p.out_stride + v] = from_f32<OUT>(y[r]);
                    }
                    if (a != kNoAdapter) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(b_empty0 + 8 * slot);
                        ++used;
                    }
                }
                if (!ok) break;
            }
            release(acc);
        }
    }
    // Everything issued is finished before shared memory and TMEM go: in a normal run the
    // epilogue has seen every tile; after an abort the copies and products in flight end by
    // themselves, and these waits are bounded like the others.
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
        if constexpr (CG == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.acc_cols << p.acc_shift));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(p.acc_cols << p.acc_shift));
    }
    if (threadIdx.x == 0 && *s_abort) flag(p.status, LP_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ host

// Map of a row-major matrix [rows][cols], read in boxes of box_cols columns (of 32, 64 or
// 128 bytes, swizzled over that width) by box_rows rows.
bool encode(CUtensorMap* map, const void* ptr, uint32_t dtype, uint64_t rows, uint64_t cols, uint64_t stride,
            uint32_t box_rows, uint32_t box_cols) {
    const EncodeFn f = encode_fn();
    if (!f) return false;
    const CUtensorMapDataType type = dtype == LP_E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : dtype == LP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t e = dtype_bytes(dtype);
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {stride * e};
    const cuuint32_t box[2] = {box_cols, box_rows}, step[2] = {1, 1};
    const CUtensorMapSwizzle swizzle = box_cols * e == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                       : box_cols * e == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                            : CU_TENSOR_MAP_SWIZZLE_32B;
    return f(map, type, 2, const_cast<void*>(ptr), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clocks of one SM that a cut takes, counted roughly: a stage of the ring costs its products
// (N / 256 x 512 clocks), its bytes at 55 a clock from L2, W's at 23.5 from HBM, or 120; a tile
// an epilogue of 8 per row and 1000, of which the last tile's is not hidden.
// Times of single CTAs and of pairs with tiles of so many rows of x, us (bf16, H = 4096; * is
// the choice):
//     48 rows on V = 152064    48: 212* | 212    32: 296
//     64 rows on V = 128256    64: 181* | 183    32: 261 | 265
//    128                      128: 177* | 179    64: 263 | 267
//    256                      256: 199 | 183*   128: 267 | 271
//   2048 rows on V = 32000    256: 312 | 294*   128: - | 523
//    256 rows on V = 4096     256: 29.3 | 29.3   64: 27.3 | 29.3   32: 45.7 (chosen: 29.3)
struct Cut {
    uint32_t cg, tile_t;
};
Cut choose_cut(uint32_t T, uint32_t V, uint32_t slices, uint32_t sms, bool adapters) {
    Cut best = {0, 0};
    double least = 0;
    for (uint32_t cg = 1; cg <= 2; ++cg) {
        const uint32_t unit = 16 * cg;
        for (uint32_t most = kMaxTileT; most >= 32; most /= 2) {
            if (T <= most / 2 && most > 32) continue;  // the same as a smaller one
            const uint32_t tiles_t = (T + most - 1) / most;
            const uint32_t tile_t = ((T + tiles_t - 1) / tiles_t + unit - 1) / unit * unit;
            if (adapters && tile_t < 32 && T > 32) continue;  // (a page of the workspace for each 32 rows)
            const double tiles = (double)((V + cg * kTileV - 1) / (cg * kTileV)) * ((T + tile_t - 1) / tile_t);
            const double units = sms / cg, waves = (double)(uint64_t)((tiles + units - 1) / units);
            const double busy = tiles < units ? tiles / units : 1.0;  // few SMs share L2's bandwidth
            double stage = 2.0 * tile_t;
            const double bytes = (kStageW + tile_t * kSliceBytes / cg) / 55.0 * (0.5 + 0.5 * busy);
            const double memory = kStageW / 23.5 * busy / tiles_t;  // W from HBM
            if (stage < bytes) stage = bytes;
            if (stage < memory) stage = memory;
            if (stage < 120) stage = 120;
            const double main = slices * stage, tail = 1000 + 8.0 * tile_t;
            const double cost = waves * (main > tail ? main : tail) + tail;
            if (best.cg == 0 || cost < least) {
                best = {cg, tile_t};
                least = cost;
            }
            if (tiles >= units) break;  // shorter tiles would only read W more often
        }
    }
    return best;
}

// B's rows go through a tensor map, as whole 16-byte pieces.
bool lora_by_tma(uint32_t rank, uint64_t adapters, uint32_t V) { return rank % 8 == 0 && adapters * V <= 0x7FFFFFFFu; }

// Blocks of rows with one adapter or two run on the tensor cores (pairs only: the tiles of fewer
// rows wait for memory, and the epilogue's arithmetic is hidden).
bool adapters_on_tensor_cores(const Cut& cut, uint32_t rank, uint64_t adapters, uint32_t V) {
    return cut.cg == 2 && rank != 0 && lora_by_tma(rank, adapters, V);
}

uint32_t slices_of(uint64_t H, uint32_t dtype) { return (uint32_t)((H * dtype_bytes(dtype) + kSliceBytes - 1) / kSliceBytes); }

struct ProjectLaunch {
    CUtensorMap w, x, b, lora_b, parts;
    ProjectParams p;
    size_t smem;
    unsigned grid;
};

template <bool FP8, typename OUT, int CG, bool LORA>
lp_status launch_project(const ProjectLaunch& l, lp_stream_t stream) {
    static std::atomic<uint64_t> smem_set;
    auto kernel = k_project<FP8, OUT, CG, !FP8 && sizeof(OUT) == 4, LORA>;
    if (!allow_smem(reinterpret_cast<const void*>(kernel), kSmemBudget, &smem_set)) return LP_ERR_CUDA;
    return launch(kernel, dim3(l.grid), kThreads, l.smem, stream, CG, l.w, l.x, l.b, l.lora_b, l.parts, l.p);
}
template <bool FP8, int CG, bool LORA>
lp_status launch_project(const ProjectLaunch& l, uint32_t out_dtype, lp_stream_t s) {
    if (out_dtype == LP_F32) return launch_project<FP8, float, CG, LORA>(l, s);
    if (out_dtype == LP_BF16) return launch_project<FP8, __nv_bfloat16, CG, LORA>(l, s);
    return launch_project<FP8, __half, CG, LORA>(l, s);
}
template <bool FP8>
lp_status launch_project(const ProjectLaunch& l, uint32_t out_dtype, uint32_t cg, lp_stream_t s) {
    if (cg == 2)
        return l.p.rank ? launch_project<FP8, 2, true>(l, out_dtype, s) : launch_project<FP8, 2, false>(l, out_dtype, s);
    return l.p.rank ? launch_project<FP8, 1, true>(l, out_dtype, s) : launch_project<FP8, 1, false>(l, out_dtype, s);
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
    if (T == 0 || V == 0) return LP_ERR_SHAPE;  // (before the pointers: an empty tensor has none)
    if (!x || !weight || !out) return LP_ERR_NULL;
    if (dtype != LP_BF16 && dtype != LP_F16 && dtype != LP_E4M3) return LP_ERR_DTYPE;
    if (out_dtype != LP_F32 && out_dtype != LP_BF16 && out_dtype != LP_F16) return LP_ERR_DTYPE;
    const bool fp8 = dtype == LP_E4M3, adapted = adapters != 0;
    if (fp8 && (!x_scale || !weight_scale)) return LP_ERR_NULL;
    if (!fp8 && (x_scale || weight_scale)) return LP_ERR_DTYPE;
    if (H == 0 || T > 0x7FFFFF00u || V > 0x7FFFFF00u || H > 0x7FFFFF00u) return LP_ERR_SHAPE;
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
        if (!aligned_to(adapter_scale, 4) || !aligned_to(adapter_ids, 4) || !aligned_to(row_offsets, 4)) return LP_ERR_SHAPE;
    } else {
        rank = 0;
    }
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < lp_head_workspace_size(rank ? T : 0, rank))
        return LP_ERR_WORKSPACE;
    const int sms = sm_count();
    if (sms == 0) return LP_ERR_CUDA;

    unsigned char* ws = static_cast<unsigned char*>(workspace);
    ProjectLaunch l = {};
    ProjectParams& p = l.p;
    p.status = reinterpret_cast<uint32_t*>(ws);
    p.x_scale = x_scale;
    p.w_scale = weight_scale;
    p.lora_b = lora_b;
    const AdapterSpace space(T, rank);
    p.groups = ws + space.groups;
    p.factor = reinterpret_cast<float*>(ws + space.factor);
    p.u = reinterpret_cast<float*>(ws + space.u);
    p.out = out;
    p.out_stride = out_stride;
    p.T = T;
    p.V = V;
    p.rank = rank;
    p.u_cols = rank_cols(rank);
    p.b_cols = part_cols(rank);
    p.lora_f16 = lora_dtype == LP_F16;
    p.lora_bytes = (uint64_t)adapters * V * rank * 2;
    p.lora_tma = lora_by_tma(rank, adapters, V);
    p.early = rank != 0;
    // How the product is cut: the rows of x into even tiles of at most 256, a multiple of 16, for
    // single CTAs or (a multiple of 32) for pairs, which read each row of x once for two tiles of
    // the vocabulary. The choice is the cheapest of a few by a rough count of clocks.
    p.slices = slices_of(H, dtype);
    const Cut cut = choose_cut(T, V, p.slices, (uint32_t)sms, rank != 0);
    const uint32_t cg = cut.cg;
    p.tile_t = cut.tile_t;
    p.tiles_t = (T + p.tile_t - 1) / p.tile_t;
    const uint64_t tiles = (uint64_t)((V + cg * kTileV - 1) / (cg * kTileV)) * p.tiles_t;
    if (tiles > 0x7FFFFFFFu) return LP_ERR_SHAPE;
    p.tiles = (uint32_t)tiles;
    p.tensor = adapters_on_tensor_cores(cut, rank, adapters, V);
    p.apart = fp8 || dtype == LP_F16;
    p.part_stride = (uint32_t)space.rows;
    p.chunk = fp8 || out_dtype != LP_F32 ? p.slices : p.tile_t <= kPromoteFewRows ? kPromoteSlices / 2 : kPromoteSlices;
    for (p.acc_cols = 32; p.acc_cols < p.tile_t; p.acc_cols *= 2) {}
    for (p.acc_shift = 1; p.acc_shift < 3 && p.acc_cols << (p.acc_shift + 1) <= 512; ++p.acc_shift) {}
    // instruction: f32 accumulator, K-major operands, M = 128 lanes a CTA, N = tile_t
    const uint32_t type = dtype == LP_BF16 ? 1u : 0u;  // kind::f16: 0 f16, 1 bf16; kind::f8f6f4: 0 e4m3
    p.idesc = (1u << 4) | (type << 7) | (type << 10) | ((p.tile_t >> 3) << 17) | ((cg * kTileV >> 4) << 24);
    const uint32_t lora_type = lora_dtype == LP_BF16 ? 1u : 0u;
    p.lora_idesc = (1u << 4) | (lora_type << 7) | (lora_type << 10) | ((cg * kTileV >> 4) << 24);  // without N
    // Shared memory: the adapters' buffers, a tile's u where that leaves four stages, and as many
    // stages as there is room for.
    const uint32_t stage_bytes = kStageW + p.tile_t / cg * kSliceBytes, slot_bytes = kTileV * p.b_cols * 2;
    const uint32_t u_bytes = p.tile_t * p.u_cols * 4;
    const uint32_t fixed = kControlBytes + (rank ? (uint32_t)sizeof(TileGroups) + (fp8 ? p.tile_t * 4 : 0) : 0);
    p.depth = rank == 0 ? 0 : rank <= 16 ? 3 : rank <= 32 ? 2 : 1;
    const uint32_t b_bytes = kShares * p.depth * slot_bytes;
    const uint32_t u_aside = kSmemBudget - fixed - b_bytes >= u_bytes + 4 * stage_bytes ? u_bytes : 0;
    p.stages = (kSmemBudget - fixed - b_bytes - u_aside) / stage_bytes;
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    p.u_smem = rank && u_aside != 0;
    l.smem = fixed + p.stages * stage_bytes + b_bytes + (p.u_smem ? u_bytes : 0);
    const uint32_t slice_cols = kSliceBytes / (uint32_t)e;
    if (!encode(&l.w, weight, dtype, V, H, weight_stride, kTileV, slice_cols) ||
        !encode(&l.x, x, dtype, T, H, x_stride, p.tile_t / cg, slice_cols))
        return LP_ERR_CUDA;
    if (rank && p.lora_tma) {
        if (!encode(&l.b, lora_b, lora_dtype, (uint64_t)adapters * V, rank, rank, kTileV, p.b_cols)) return LP_ERR_CUDA;
    }
    if (p.tensor) {
        if (!encode(&l.lora_b, lora_b, lora_dtype, (uint64_t)adapters * V, rank, rank, kTileV, 64) ||
            !encode(&l.parts, ws + space.parts, lora_dtype, part_rows(rank) * space.rows, 64, 64, kBlock / cg, 64))
            return LP_ERR_CUDA;
    }
    if (rank) {
        ShrinkParams q = {};
        q.x = x;
        q.x_scale = x_scale;
        q.lora_a = lora_a;
        q.adapter_scale = adapter_scale;
        q.adapter_ids = adapter_ids;
        q.row_offsets = row_offsets;
        q.u = const_cast<float*>(p.u);
        q.groups = ws + space.groups;
        q.factor = reinterpret_cast<float*>(ws + space.factor);
        q.parts = reinterpret_cast<uint16_t*>(ws + space.parts);
        q.tile_t = p.tile_t;
        q.tensor = p.tensor;
        q.apart = p.apart;
        q.part_stride = p.part_stride;
        q.lora_f16 = p.lora_f16;
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
    const uint32_t units = (uint32_t)sms / cg;  // CTAs, or pairs
    l.grid = cg * (p.tiles < units ? p.tiles : units);
    return fp8 ? launch_project<true>(l, out_dtype, cg, stream) : launch_project<false>(l, out_dtype, cg, stream);
}

extern "C" lp_status lp_head_project_cut(uint32_t T, uint32_t H, uint32_t V, uint32_t dtype, uint32_t adapters,
                                         uint32_t rank, uint32_t sms, uint32_t* ctas, uint32_t* rows,
                                         uint32_t* on_tensor_cores) {
    if (!ctas || !rows || !on_tensor_cores) return LP_ERR_NULL;
    if (dtype != LP_BF16 && dtype != LP_F16 && dtype != LP_E4M3) return LP_ERR_DTYPE;
    if (T == 0 || H == 0 || V == 0 || T > 0x7FFFFF00u || V > 0x7FFFFF00u || H > 0x7FFFFF00u || rank > LP_MAX_RANK)
        return LP_ERR_SHAPE;
    if (adapters == 0) rank = 0;
    if (sms == 0) sms = (uint32_t)sm_count();
    if (sms < 2) return LP_ERR_CUDA;
    const Cut cut = choose_cut(T, V, slices_of(H, dtype), sms, rank != 0);
    *ctas = cut.cg;
    *rows = cut.tile_t;
    *on_tensor_cores = adapters_on_tensor_cores(cut, rank, adapters, V);
    return LP_OK;
}
