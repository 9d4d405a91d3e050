// Rows in microscaled 4-bit floating point (include/lp_head.h): quantised in blocks of 16 or
// 32, and read back as values, all of them or those that an index picks.
//
// Quantising is one pass: a thread holds groups of eight neighbouring elements in registers, a
// block is two or four neighbouring lanes, and (blocks of 16) the row's largest magnitude is
// reduced before the first scale is formed. Scales are powers of two or have four significant
// bits, so every quotient below is either exact or rounded once, and a value half way between two
// codes goes where the formula says. Bound by HBM.
#include "lp_head_common.h"

namespace {

using namespace lph;

constexpr int kVec = 8;  // elements of a group: 16 bytes of 16-bit input, 4 bytes of codes

struct QuantParams {
    const void* x;
    unsigned char* codes;
    unsigned char* scales;
    float* row_scale;
    uint64_t x_stride, codes_stride;
    uint32_t T, H, col_tiles;
    uint32_t aligned;  // rows of x begin on 16 bytes
};

// Byte of the scale of block `col` of row `row`: tiles of 128 rows by 4 blocks, each
// [row % 32][row / 32 % 4][col % 4].
__device__ __forceinline__ uint64_t scale_at(uint32_t row, uint32_t col, uint32_t col_tiles) {
    return ((uint64_t)(row >> 7) * col_tiles + (col >> 2)) * 512 + (row & 31) * 16 + (row >> 5 & 3) * 4 + (col & 3);
}

// Eight elements as floats.
__device__ __forceinline__ void load8(const float* p, bool aligned, float (&v)[kVec]) {
    if (aligned) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = p[i];
    }
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool aligned, float (&v)[kVec]) {
    if (aligned) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = unpack2(u[i], T());
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = to_f32(p[i]);
    }
}

__device__ __forceinline__ uint32_t codes_of(const float (&q)[kVec]) {  // nearest even, saturated, low half first
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r) : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}

__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // e in -126..127

// BLOCK: elements of a scale. TPR threads take a row, U groups each.
template <typename T, int BLOCK, int TPR, int U, int CTA>
__global__ void __launch_bounds__(CTA) k_quantize4(const QuantParams p) {
    constexpr int kRows = CTA / TPR, kLanes = BLOCK / kVec;  // lanes that share a scale
    constexpr int kWarps = TPR / 32;
    [[maybe_unused]] __shared__ float s_max[CTA / 32];
    pdl_trigger();
    pdl_wait();
    const uint32_t r = threadIdx.x / TPR, t = threadIdx.x % TPR;
    const uint32_t row = blockIdx.x * kRows + r, groups = p.H / kVec, blocks = p.H / BLOCK;
    const bool live = row < p.T;
    const T* x = static_cast<const T*>(p.x) + (uint64_t)(live ? row : 0) * p.x_stride;
    float v[U][kVec];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t g = u * TPR + t;
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[u][i] = 0.f;
        if (live && g < groups) load8(x + (uint64_t)g * kVec, p.aligned, v[u]);
    }
    float top[U];  // of the block that a group is part of
#pragma unroll
    for (int u = 0; u < U; ++u) {
        top[u] = 0.f;
#pragma unroll
        for (int i = 0; i < kVec; ++i) top[u] = max_nan(top[u], fabsf(v[u][i]));
#pragma unroll
        for (int m = 1; m < kLanes; m *= 2) top[u] = max_nan(top[u], __shfl_xor_sync(0xFFFFFFFFu, top[u], m));
    }
    int e = 0;  // the row's scale is 2^e
    bool finite = true;
    if constexpr (BLOCK == 16) {
        float m = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) m = max_nan(m, top[u]);
#pragma unroll
        for (int k = 16; k > 0; k /= 2) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, k));
        if constexpr (kWarps > 1) {
            if ((threadIdx.x & 31) == 0) s_max[threadIdx.x / 32] = m;
            __syncthreads();
            m = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) m = max_nan(m, s_max[r * kWarps + k]);
        }
        finite = m < __uint_as_float(0x7F800000u);  // (false for NaN)
        // the smallest power of two r with m <= 6 * 448 r = 1.3125 * 2^11 r, at least 2^-100
        const uint32_t bits = __float_as_uint(m);
        const int above = (int)(bits >> 23) - 127;  // m = f 2^above, 1 <= f < 2 (subnormal m: far below 2^-100)
        e = max(above - 11 + ((bits & 0x7FFFFFu) > 0x280000u), -100);
        if (t == 0 && live) p.row_scale[row] = finite ? power_of_two(e) : __uint_as_float(0x7FC00000u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t g = u * TPR + t;
        uint32_t byte;
        float q[kVec];
        if constexpr (BLOCK == 16) {
            const float inv = power_of_two(-e);
            const float want = __fdiv_rn(top[u] * inv, 6.f);
            byte = finite ? (uint32_t)__nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3) : 0x7Fu;
            // 1 / scale rounded, and quotients corrected by their remainder: rounded once
            const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
            const float r1 = byte ? __frcp_rn(s) : 0.f;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float y = v[u][i] * inv, a = y * r1;
                q[i] = fmaf(fmaf(-a, s, y), r1, a);
            }
        } else {
            const uint32_t bits = __float_as_uint(top[u]);
            // floor(log2) - 2 of the largest, biased by 127: its exponent field less 2 (subnormals: 0)
            const int b = max((int)(bits >> 23) - 2, 0);
            byte = top[u] < __uint_as_float(0x7F800000u) ? (uint32_t)b : 0xFFu;
            const float inv = power_of_two(127 - b);
#pragma unroll
            for (int i = 0; i < kVec; ++i) q[i] = v[u][i] * inv;
        }
        if (live && g < groups) {
            *reinterpret_cast<uint32_t*>(p.codes + (uint64_t)row * p.codes_stride + (uint64_t)g * (kVec / 2)) = codes_of(q);
            if (g % kLanes == 0) p.scales[scale_at(row, g / kLanes, p.col_tiles)] = (unsigned char)byte;
        }
    }
    // zeros around the scales: past a row's blocks, and in the rows past the last
    for (uint32_t c = (live ? blocks : 0) + t; c < p.col_tiles * 4; c += TPR) p.scales[scale_at(row, c, p.col_tiles)] = 0;
}

template <typename T, int BLOCK>
lp_status launch_quantize(const QuantParams& p, lp_stream_t stream) {
    const uint32_t groups = p.H / kVec, rows = (p.T + 127) / 128 * 128;
    if (groups <= 128)
        return launch(k_quantize4<T, BLOCK, 32, 4, 128>, dim3(rows / 4), 128, 0, stream, 1, p);
    if (groups <= 512) return launch(k_quantize4<T, BLOCK, 128, 4, 128>, dim3(rows), 128, 0, stream, 1, p);
    if (groups <= 1024) return launch(k_quantize4<T, BLOCK, 256, 4, 256>, dim3(rows), 256, 0, stream, 1, p);
    return launch(k_quantize4<T, BLOCK, 512, 8, 512>, dim3(rows), 512, 0, stream, 1, p);
}
template <typename T>
lp_status launch_quantize(const QuantParams& p, uint32_t block, lp_stream_t stream) {
    return block == 16 ? launch_quantize<T, 16>(p, stream) : launch_quantize<T, 32>(p, stream);
}

struct DequantParams {
    const unsigned char* codes;
    const unsigned char* scales;
    const float* row_scale;
    const uint32_t* rows;
    void* out;
    uint32_t* status;
    uint64_t codes_stride, out_stride;
    uint32_t V, n, H, col_tiles;
    uint32_t aligned;  // out's rows begin on 16 bytes
};

template <typename T>
__device__ __forceinline__ void store8(T* p, bool aligned, const float (&v)[kVec]) {
    if (!aligned) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) p[i] = from_f32<T>(v[i]);
    } else if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()), pack2(v[4], v[5], T()),
                                                  pack2(v[6], v[7], T()));
    }
}

constexpr int kDequantThreads = 128;

// A CTA takes a piece of a row: kDequantThreads groups of eight codes, four times.
template <typename T, int BLOCK>
__global__ void __launch_bounds__(kDequantThreads) k_dequantize4(const DequantParams p) {
    pdl_trigger();
    pdl_wait();
    const uint32_t o = blockIdx.x, groups = p.H / kVec;
    const uint32_t row = p.rows ? p.rows[o] : o;
    T* out = static_cast<T*>(p.out) + (uint64_t)o * p.out_stride;
    const bool bad = row >= p.V;
    if (bad && threadIdx.x == 0 && blockIdx.y == 0) flag(p.status, LP_ERR_OFFSETS);
    const float nan = __uint_as_float(0x7FC00000u);
    const float rs = bad ? nan : p.row_scale ? p.row_scale[row] : 1.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t g = (blockIdx.y * 4 + k) * kDequantThreads + threadIdx.x;
        if (g >= groups) return;
        float v[kVec];
        if (bad) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[i] = nan;
        } else {
            const uint32_t c = *reinterpret_cast<const uint32_t*>(p.codes + (uint64_t)row * p.codes_stride + (uint64_t)g * 4);
            const uint32_t byte = p.scales[scale_at(row, g * kVec / BLOCK, p.col_tiles)];
            float s;
            if constexpr (BLOCK == 16) s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
            else s = byte == 255 ? nan : byte ? power_of_two((int)byte - 127) : __uint_as_float(0x00400000u);  // 2^-127
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                // the three bits below the sign: exponent and mantissa of 0, 0.5, 1, 1.5, 2, 3, 4, 6
                const uint32_t m = c >> (4 * i) & 7, sign = (c >> (4 * i + 3) & 1) << 31;
                const float level = __uint_as_float((m < 2 ? m * 0x3F000000u : ((m + 252u) << 22)) | sign);
                v[i] = level * s * rs;  // (the first product is exact)
            }
        }
        store8(out + (uint64_t)g * kVec, p.aligned, v);
    }
}

template <typename T>
lp_status launch_dequantize(const DequantParams& p, uint32_t block, lp_stream_t stream) {
    const dim3 grid(p.n, (p.H / kVec + 4 * kDequantThreads - 1) / (4 * kDequantThreads));
    return block == 16 ? launch(k_dequantize4<T, 16>, grid, kDequantThreads, 0, stream, 1, p)
                       : launch(k_dequantize4<T, 32>, grid, kDequantThreads, 0, stream, 1, p);
}

bool block_ok(uint32_t block) { return block == 16 || block == 32; }

}  // namespace

extern "C" size_t lp_head_fp4_scale_bytes(uint32_t rows, uint32_t H, uint32_t block) {
    if (!block_ok(block)) return 0;
    const uint64_t blocks = ((uint64_t)H + block - 1) / block;
    return (size_t)(((uint64_t)rows + 127) / 128 * ((blocks + 3) / 4) * 512);
}

extern "C" lp_status lp_head_quantize4(const void* x, uint32_t dtype, uint32_t T, uint32_t H, uint64_t x_stride,
                                       uint32_t block, void* codes, uint64_t codes_stride, void* scales,
                                       float* row_scale, lp_stream_t stream) {
    if (T == 0 || H == 0) return LP_ERR_SHAPE;
    if (!x || !codes || !scales) return LP_ERR_NULL;
    if (dtype != LP_F32 && dtype != LP_BF16 && dtype != LP_F16) return LP_ERR_DTYPE;
    if (!block_ok(block) || H % 32 || H > LP_MAX_HIDDEN || T > 0x7FFFFF00u) return LP_ERR_SHAPE;
    if ((block == 16) != (row_scale != nullptr)) return row_scale ? LP_ERR_DTYPE : LP_ERR_NULL;
    if (x_stride < H || codes_stride < H / 2 || codes_stride % 16) return LP_ERR_SHAPE;
    const size_t e = dtype_bytes(dtype);
    if (!aligned_to(x, e) || !aligned_to(codes, 16) || !aligned_to(scales, 16) || !aligned_to(row_scale, 4)) return LP_ERR_SHAPE;
    QuantParams p = {};
    p.x = x;
    p.codes = static_cast<unsigned char*>(codes);
    p.scales = static_cast<unsigned char*>(scales);
    p.row_scale = row_scale;
    p.x_stride = x_stride;
    p.codes_stride = codes_stride;
    p.T = T;
    p.H = H;
    p.col_tiles = (H / block + 3) / 4;
    p.aligned = aligned_to(x, 16) && (T == 1 || x_stride * e % 16 == 0);
    if (dtype == LP_F32) return launch_quantize<float>(p, block, stream);
    if (dtype == LP_BF16) return launch_quantize<__nv_bfloat16>(p, block, stream);
    return launch_quantize<__half>(p, block, stream);
}

extern "C" lp_status lp_head_dequantize4(const void* codes, uint64_t codes_stride, const void* scales,
                                         const float* row_scale, uint32_t V, uint32_t H, uint32_t block,
                                         const uint32_t* rows, uint32_t n, void* out, uint32_t out_dtype,
                                         uint64_t out_stride, void* workspace, size_t workspace_bytes,
                                         lp_stream_t stream) {
    if (V == 0 || H == 0 || n == 0 || (!rows && n != V)) return LP_ERR_SHAPE;
    if (!codes || !scales || !out) return LP_ERR_NULL;
    if (out_dtype != LP_F32 && out_dtype != LP_BF16 && out_dtype != LP_F16) return LP_ERR_DTYPE;
    if (!block_ok(block) || H % 32 || H > LP_MAX_HIDDEN || V > 0x7FFFFF00u || n > 0x7FFFFF00u) return LP_ERR_SHAPE;
    if (codes_stride < H / 2 || codes_stride % 16 || out_stride < H) return LP_ERR_SHAPE;
    const size_t e = dtype_bytes(out_dtype);
    if (!aligned_to(codes, 16) || !aligned_to(scales, 16) || !aligned_to(row_scale, 4) || !aligned_to(rows, 4) ||
        !aligned_to(out, e))
        return LP_ERR_SHAPE;
    if (rows && (!workspace || workspace_bytes < kHeaderBytes)) return LP_ERR_WORKSPACE;
    if (workspace && !aligned_to(workspace, 256)) return LP_ERR_WORKSPACE;
    DequantParams p = {};
    p.codes = static_cast<const unsigned char*>(codes);
    p.scales = static_cast<const unsigned char*>(scales);
    p.row_scale = row_scale;
    p.rows = rows;
    p.out = out;
    p.status = static_cast<uint32_t*>(workspace);
    p.codes_stride = codes_stride;
    p.out_stride = out_stride;
    p.V = V;
    p.n = n;
    p.H = H;
    p.col_tiles = (H / block + 3) / 4;
    p.aligned = aligned_to(out, 16) && (n == 1 || out_stride * e % 16 == 0);
    if (out_dtype == LP_F32) return launch_dequantize<float>(p, block, stream);
    if (out_dtype == LP_BF16) return launch_dequantize<__nv_bfloat16>(p, block, stream);
    return launch_dequantize<__half>(p, block, stream);
}
