// What the projection's two kernels share: the layout of a call's workspace and the
// per-tile lists of adapters that the first kernel writes for the second.
#pragma once

#include "lp_head_common.h"

namespace lph {

constexpr uint32_t kMaxTileT = 256;  // rows of x of a tile
constexpr uint32_t kItemRows = 32;
constexpr uint32_t kMaxItems = kMaxTileT + kMaxTileT / kItemRows;
constexpr uint32_t kBlock = 32;      // rows of a block: what one epilogue pass takes
constexpr uint32_t kNoAdapter = 0xFFFFFFFFu;

// One tile of rows, in blocks of 32. Where all rows of a block have one adapter, its part of
// the product runs on the tensor cores: in pass 0, which adds to the product's own accumulator,
// or, where that cannot be (`apart`), in pass 1, which has one of its own. Pass 1 also takes the
// two adapters of blocks that have two, or one and rows without: the epilogue adds the rows that
// have the adapter. The second adapter's sums lie in columns of a block that is not in the pass.
// The rows of other blocks (and where no such column is left) are grouped by adapter, those
// without one last, and cut into items of at most kItemRows rows of one adapter, which the
// epilogue multiplies itself.
// (Zeroing u in other adapters' rows instead would let an infinity in one adapter's B become
// NaN, 0 x inf, in the rows of others.)
constexpr uint32_t kBlocks = kMaxTileT / kBlock;
constexpr uint32_t kMaxRuns = 2 * kBlocks;
struct TileGroups {
    uint32_t items;
    uint32_t listed;             // bit per block: its rows are in items
    uint32_t runs;
    uint32_t blocks;             // bit per block: it is in pass 1
    uint32_t second;             // bit per block: with two adapters
    uint32_t place;              // 4 bits per block: the block whose columns hold the second one's sums
    uint32_t unused[2];
    uint32_t rows[2][kBlocks];   // the block's rows that have its first, its second adapter, a bit each
    uint2 run[kMaxRuns];         // neighbouring blocks with one adapter in a pass, in the order of the
                                 // passes: x = place of the sums << 24 | pass << 16 | first block << 8
                                 // | blocks, y = adapter
    uint32_t item[kMaxItems];    // adapter of item k, kNoAdapter for rows without one
    uint8_t start[kMaxItems];    // item k holds order[start[k] ... start[k] + size[k] - 1]
    uint8_t size[kMaxItems];
    uint8_t order[kMaxTileT];    // row within the tile
};
constexpr size_t kGroupBytes = 2560;  // of one tile in the workspace
static_assert(sizeof(TileGroups) % 16 == 0 && sizeof(TileGroups) <= kGroupBytes, "read as 16-byte words");

// u of a row for the tensor cores: three 16-bit parts (the value rounded towards zero, what that
// left, rounded the same way, and the rest), each padded to b_cols columns, packed into rows of 64
// columns.
__host__ __device__ constexpr uint32_t rank_cols(uint32_t rank) { return (rank + 15) & ~15u; }
__host__ __device__ constexpr uint32_t part_cols(uint32_t rank) { return rank <= 16 ? 16 : rank <= 32 ? 32 : 64; }
__host__ __device__ constexpr uint32_t part_rows(uint32_t rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : 3; }

// The workspace: header, a page a tile of rows (of 32 at least, or all rows), a factor a row, u
// (f32, padded to a multiple of 16), and u as parts ([part_rows][rows][64]).
struct AdapterSpace {
    size_t rows, groups, factor, u, parts, bytes;
    AdapterSpace(uint32_t T, uint32_t rank) {
        const size_t tiles = ((size_t)T + kBlock - 1) / kBlock;
        rows = ((size_t)T + kMaxTileT - 1) / kMaxTileT * kMaxTileT;
        groups = kHeaderBytes;
        factor = groups + tiles * kGroupBytes;
        u = factor + rows * 4;
        parts = u + rows * rank_cols(rank) * 4;
        bytes = rank == 0 ? kHeaderBytes : parts + (size_t)part_rows(rank) * rows * 128;
    }
};

struct ShrinkParams {
    const void* x;
    const float* x_scale;
    const void* lora_a;           // [A][rank][H]
    const float* adapter_scale;   // [A] or NULL
    const int32_t* adapter_ids;   // [B]
    const uint32_t* row_offsets;  // [B+1] or NULL
    unsigned char* groups;
    float* factor;
    float* u;
    uint16_t* parts;
    uint32_t* status;
    uint64_t x_stride;
    uint32_t T, H, B, adapters, rank;
    uint32_t tile_t;              // rows of a tile
    uint32_t part_stride;         // rows of u's parts
    uint32_t tensor;              // blocks of one adapter run on the tensor cores (u's parts are wanted)
    uint32_t apart;               // none in the product's own accumulator (pass 0)
    uint32_t lora_f16;
};

lp_status launch_shrink(const ShrinkParams& p, uint32_t dtype, uint32_t lora_dtype, lp_stream_t stream);

}  // namespace lph
