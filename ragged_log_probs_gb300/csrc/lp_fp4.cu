// Rows in microscaled 4-bit floating point (include/lp_head.h): quantised in blocks of 16 or
// 32, and read back as values, all of them or those that an index picks.
//
// Quantising is one pass: a thread holds groups of sixteen neighbouring elements in registers, a
// block is one or two neighbouring lanes, and (blocks of 16) the row's largest magnitude is
// reduced before the first scale is formed. Scales are powers of two or have four significant
// bits, so every quotient below is either exact or rounded once, and a value half way between two
// codes goes where the formula says. Bound by HBM, and for blocks of 16 nearly as much by the
// quotients (three operations each): 32000 rows of 4096 bf16 in blocks of 16 70 us (4.8 TB/s, 71 % of
// a copy's rate), of 32 51 (6.5 TB/s). Read back, 32000 such rows 60 us (5.6 TB/s), bound by HBM.
#include "lp_head_common.h"

namespace {

using namespace lph;

constexpr int kVec = 16;  // elements of a group: 8 bytes of codes

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

// Sixteen elements as floats.
__device__ __forceinline__ void load16(const float* p, bool aligned, float (&v)[kVec]) {
    if (aligned) {
#pragma unroll
        for (int i = 0; i < kVec; i += 4) {
            const float4 a = *reinterpret_cast<const float4*>(p + i);
            v[i] = a.x; v[i + 1] = a.y; v[i + 2] = a.z; v[i + 3] = a.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = p[i];
    }
}
template <typename T>
__device__ __forceinline__ void load16(const T* p, bool aligned, float (&v)[kVec]) {
    if (aligned) {
#pragma unroll
        for (int k = 0; k < kVec; k += 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + k);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = unpack2(u[i], T());
                v[k + 2 * i] = f.x;
                v[k + 2 * i + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = to_f32(p[i]);
    }
}

__device__ __forceinline__ uint32_t codes_of(const float* q) {  // of eight: nearest even, saturated, low half first
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
        if (live && g < groups) load16(x + (uint64_t)g * kVec, p.aligned, v[u]);
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
            const float want = __fdiv_rn(top[u] * power_of_two(-e), 6.f);
            byte = finite ? (uint32_t)__nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3) : 0x7Fu;
            // The quotient by s = scale * 2^e: by the rounded 1 / s, and corrected by its remainder: rounded once.
            const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
            const float whole = s * power_of_two(e), inv = byte ? __frcp_rn(s) * power_of_two(-e) : 0.f;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const float a = v[u][i] * inv;
                q[i] = fmaf(fmaf(-a, whole, v[u][i]), inv, a);
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
            *reinterpret_cast<uint2*>(p.codes + (uint64_t)row * p.codes_stride + (uint64_t)g * (kVec / 2)) = make_uint2(codes_of(q), codes_of(q + 8));
            if (g % kLanes == 0) p.scales[scale_at(row, g / kLanes, p.col_tiles)] = (unsigned char)byte;
        }
    }
    // zeros around the scales: past a row's blocks, and in the rows past the last
    for (uint32_t c = (live ? blocks : 0) + t; c < p.col_tiles * 4; c += TPR) p.scales[scale_at(row, c, p.col_tiles)] = 0;
}

template <typename T, int BLOCK>
lp_status launch_quantize(const QuantParams& p, lp_stream_t stream) {
    const uint32_t groups = p.H / kVec, rows = (p.T + 127) / 128 * 128;
    if (groups <= 64) return launch(k_quantize4<T, BLOCK, 32, 2, 128>, dim3(rows / 4), 128, 0, stream, 1, p);
    // one group a thread (32000 rows of 4096 bf16: 70 us and, blocks of 32, 51; two a thread 73 and 56, a row a
    // warp 77 and 67)
    if (groups <= 256) return launch(k_quantize4<T, BLOCK, 256, 1, 256>, dim3(rows), 256, 0, stream, 1, p);
    if (groups <= 512) return launch(k_quantize4<T, BLOCK, 512, 1, 512>, dim3(rows), 512, 0, stream, 1, p);
    return launch(k_quantize4<T, BLOCK, 512, 4, 512>, dim3(rows), 512, 0, stream, 1, p);
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
__device__ __forceinline__ void store16(T* p, bool aligned, const float (&v)[kVec]) {
    if (!aligned) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) p[i] = from_f32<T>(v[i]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < kVec; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; i += 8)
            *reinterpret_cast<uint4*>(p + i) = make_uint4(pack2(v[i], v[i + 1], T()), pack2(v[i + 2], v[i + 3], T()),
                                                          pack2(v[i + 4], v[i + 5], T()), pack2(v[i + 6], v[i + 7], T()));
    }
}
// The levels of eight codes, as pairs of halves.
__device__ __forceinline__ void levels_of(uint32_t codes, __half2 (&l)[4]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(l);
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(codes));
}

constexpr uint32_t kDequantThreads = 256, kDequantItems = 2 * kDequantThreads;  // groups of a CTA

// A CTA takes kDequantItems groups: of a row's piece, or of several short rows.
template <typename T, int BLOCK>
__global__ void __launch_bounds__(kDequantThreads) k_dequantize4(const DequantParams p) {
    pdl_trigger();
    pdl_wait();
    const uint32_t groups = p.H / kVec, several = kDequantItems / groups;  // rows of a CTA, 0: pieces of one
    const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (uint32_t k = 0; k < kDequantItems / kDequantThreads; ++k) {
        uint32_t o = blockIdx.x, g = blockIdx.y * kDequantItems + k * kDequantThreads + threadIdx.x;
        if (several) {
            const uint32_t r = g / groups;
            if (r >= several) return;
            o = o * several + r;
            g -= r * groups;
        }
        if (o >= p.n || g >= groups) return;
        const uint32_t row = p.rows ? p.rows[o] : o;
        float v[kVec];
        if (row >= p.V) {
            if (g == 0) flag(p.status, LP_ERR_OFFSETS);
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[i] = nan;
        } else {
            const uint2 c = *reinterpret_cast<const uint2*>(p.codes + (uint64_t)row * p.codes_stride + (uint64_t)g * 8);
            const uint32_t byte = p.scales[scale_at(row, g * kVec / BLOCK, p.col_tiles)];
            const float rs = p.row_scale ? p.row_scale[row] : 1.f;
            __half2 l[8];
            levels_of(c.x, reinterpret_cast<__half2(&)[4]>(l[0]));
            levels_of(c.y, reinterpret_cast<__half2(&)[4]>(l[4]));
            float s = 1.f;
            if constexpr (BLOCK == 16) {  // six bits and exponents from -10 to 11: exact in f16
                const __half2 s2 = __half2half2(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
#pragma unroll
                for (int i = 0; i < 8; ++i) l[i] = __hmul2(l[i], s2);
            } else {
                s = byte == 255 ? nan : byte ? power_of_two((int)byte - 127) : __uint_as_float(0x00400000u);  // 2^-127
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = __half22float2(l[i]);
                v[2 * i] = BLOCK == 16 ? f.x * rs : f.x * s * rs;  // (the product with s is exact)
                v[2 * i + 1] = BLOCK == 16 ? f.y * rs : f.y * s * rs;
            }
        }
        store16(static_cast<T*>(p.out) + (uint64_t)o * p.out_stride + (uint64_t)g * kVec, p.aligned, v);
    }
}

template <typename T>
lp_status launch_dequantize(const DequantParams& p, uint32_t block, lp_stream_t stream) {
    const uint32_t groups = p.H / kVec, several = kDequantItems / groups;
    const dim3 grid(several ? (p.n + several - 1) / several : p.n, several ? 1 : (groups + kDequantItems - 1) / kDequantItems);
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
