// Final norm of a model's head: residual addition, root-mean-square norm, and an output
// in the input's type, f32, or e4m3 with one f32 scale a row (include/lp_head.h).
//
// One pass over the data. A row stays in registers between its two uses: h = x + residual
// is formed in f32 while it is loaded, the row's sum of h^2 and largest |h w| are reduced
// together (|y| is largest where |h w| is: the factor 1/rms is common to the row), and the
// output is written from the registers. Bound by HBM: every element is read once and
// written once. The largest LP_MAX_HIDDEN row is 1024 threads x 4 vectors of 8.
#include "lp_head_common.h"

namespace {

using namespace lph;

constexpr int kVec = 8;         // elements a thread handles together
constexpr int kWarpRowVecs = 128;  // rows of up to this many vectors (1024 elements): a warp each
constexpr int kWarpRows = 4;    // rows (warps) per CTA then

struct NormParams {
    const void* x;
    const void* residual;
    const void* weight;
    const uint32_t* rows;
    void* out;
    float* out_scale;
    void* residual_out;
    uint32_t* status;
    uint64_t x_stride, residual_stride, out_stride, residual_out_stride;
    uint32_t T, n, H;
    uint32_t shift;       // groups of eight follow the output's boundaries (kShifted)
    uint32_t weight_f32;  // weight is f32 whatever the rows' type
    float eps;
};

// Where a thread's eight elements lie. kAligned: neighbours, all in the row, on a 16-byte
// boundary. Rows at other boundaries: kShifted, neighbours from any element on, also before the
// row's first, or kStrided, every `step`-th, so that a warp's lanes read neighbours. The first
// reads the aligned 16-byte words that hold the eight and shifts, which takes fewer loads and
// costs more at a row's ends: 333 rows of 5001 f16 7.3 us, strided 9.0; 10757 of 6622 bf16 92 and
// 107; but 8746 of 390, a warp each, 14.5 and 10.5.
enum Layout { kAligned, kShifted, kStrided };

// Eight elements out of their words.
__device__ __forceinline__ void widen(const uint32_t (&w)[8], float (&v)[kVec], float) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = __uint_as_float(w[i]);
}
template <typename T>
__device__ __forceinline__ void widen(const uint32_t (&w)[8], float (&v)[kVec], T) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(w[i], T());
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void read16(const void* p, uint32_t* w) {
    const uint4 a = *static_cast<const uint4*>(p);
    w[0] = a.x;
    w[1] = a.y;
    w[2] = a.z;
    w[3] = a.w;
}

// The eight elements from e on, zero where the row of H has none.
template <typename T, Layout L>
__device__ __forceinline__ void load8(const T* p, int e, int step, int H, float (&v)[kVec]) {
    constexpr int kIn16 = 16 / sizeof(T), kWords = 2 * sizeof(T);  // 32-bit words of the eight
    const int m = L == kShifted ? (int)((reinterpret_cast<uintptr_t>(p + e) & 15) / sizeof(T)) : 0;
    if (L == kAligned || (L == kShifted && e - m >= 0 && e - m + kVec + (m ? kIn16 : 0) <= H)) {
        uint32_t w[12];
        const T* q = p + e - m;
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) read16(q + i * kIn16, w + 4 * i);
        if (m) {
            read16(q + kVec, w + kWords);
            if (sizeof(T) == 2) {
                if (m & 4)
#pragma unroll
                    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
                if (m & 2)
#pragma unroll
                    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
                if (m & 1)
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
            } else {
                if (m & 2)
#pragma unroll
                    for (int i = 0; i < 10; ++i) w[i] = w[i + 2];
                if (m & 1)
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = w[i + 1];
            }
        }
        uint32_t eight[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) eight[i] = i < kWords ? w[i] : 0u;
        widen(eight, v, T());
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int at = L == kStrided ? e + i * step : e + i;
            v[i] = at >= 0 && at < H ? to_f32(p[at]) : 0.f;
        }
    }
}

template <typename T, Layout L>
__device__ __forceinline__ void store8(T* p, int e, int step, int H, const float (&v)[kVec]) {
    if (L == kAligned || (L == kShifted && e >= 0 && e + kVec <= H && (reinterpret_cast<uintptr_t>(p + e) & 15) == 0)) {
        p += e;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()),
                                                      pack2(v[4], v[5], T()), pack2(v[6], v[7], T()));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int at = L == kStrided ? e + i * step : e + i;
            if (at >= 0 && at < H) p[at] = from_f32<T>(v[i]);
        }
    }
}

template <Layout L>
__device__ __forceinline__ void store8_e4m3(uint8_t* p, int e, int step, int H, const float (&v)[kVec]) {
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // round to nearest even, saturating; NaN stays NaN
        h[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    if (L == kAligned || (L == kShifted && e >= 0 && e + kVec <= H && (reinterpret_cast<uintptr_t>(p + e) & 7) == 0)) {
        *reinterpret_cast<uint2*>(p + e) = make_uint2(h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16));
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int at = L == kStrided ? e + i * step : e + i;
            if (at >= 0 && at < H) p[at] = (uint8_t)(h[i / 2] >> (8 * (i & 1)));
        }
    }
}

// One row by `threads` threads (a warp, or the CTA when WARP is false), this thread `tid`.
template <typename T, typename O, Layout L, bool WARP, int NV>
__device__ __forceinline__ void norm_row(const NormParams& p, uint32_t o, int tid, int threads, float (*red)[2]) {
    constexpr bool kQuant = sizeof(O) == 1;
    uint32_t i = o;
    bool bad = false;
    if (p.rows) {
        i = p.rows[o];
        bad = i >= p.T;
        if (bad) {
            i = 0;
            if (tid == 0) flag(p.status, LP_ERR_OFFSETS);
        }
    }
    const T* x = static_cast<const T*>(p.x) + (uint64_t)i * p.x_stride;
    const T* r = p.residual ? static_cast<const T*>(p.residual) + (uint64_t)i * p.residual_stride : nullptr;
    const int H = (int)p.H;
    const auto load_weight = [&](int e, float (&g)[kVec]) {
        if (sizeof(T) < 4 && !p.weight_f32) load8<T, L>(static_cast<const T*>(p.weight), e, threads, H, g);
        else load8<float, L>(static_cast<const float*>(p.weight), e, threads, H, g);
    };
    O* out = static_cast<O*>(p.out) + (uint64_t)o * p.out_stride;
    // Where the thread's k-th eight begin. Shifted groups follow the output's boundaries (which in
    // one layout are those of x and residual too).
    const int shift = L == kShifted && p.shift ? (int)(reinterpret_cast<uintptr_t>(out) / sizeof(O) % kVec) : 0;
    const auto begin = [&](int k) { return L == kStrided ? tid + k * kVec * threads : (tid + k * threads) * kVec - shift; };
    float h[NV][kVec];
    float sum = 0.f, top = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = begin(k);
        if (e < H) load8<T, L>(x, e, threads, H, h[k]);
    }
    if (r) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = begin(k);
            float v[kVec];
            if (e < H) {
                load8<T, L>(r, e, threads, H, v);
#pragma unroll
                for (int j = 0; j < kVec; ++j) h[k][j] += v[j];
            }
        }
    }
    if (bad) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
            for (int j = 0; j < kVec; ++j) h[k][j] = __int_as_float(0x7fffffff);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = begin(k);
        if (e < H) {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                sum = fmaf(h[k][j], h[k][j], sum);
            if constexpr (kQuant) {
                float g[kVec];
                load_weight(e, g);
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    top = max_nan(top, fabsf(h[k][j] * g[j]));
            }
        }
    }
    const auto over_row = [&](float& sum, float& top) {  // every thread gets the same bits
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            if constexpr (kQuant) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        }
        if constexpr (!WARP) {
            const int warp = tid >> 5, lane = tid & 31, warps = threads >> 5;
            if (lane == 0) {
                red[warp][0] = sum;
                red[warp][1] = top;
            }
            __syncthreads();
            sum = lane < warps ? red[lane][0] : 0.f;
            top = lane < warps ? red[lane][1] : 0.f;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
                if constexpr (kQuant) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            }
        }
    };
    over_row(sum, top);
    float mean = sum / (float)p.H + p.eps, inv = rsqrtf(mean);
    T* kept = p.residual_out ? static_cast<T*>(p.residual_out) + (uint64_t)o * p.residual_out_stride : nullptr;
    // A row whose squares or products h w leave f32 (or hold a NaN or an infinity): once more, of
    // h times a power of two that brings them back, with the largest |y| itself.
    const bool large = !(mean < 0x1p120f), small = mean < 0x1p-90f;
    if (large || small || (kQuant && sum > 0.f && !(top > 0x1p-100f && top < 0x1p120f))) {
        if (kept) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (begin(k) < H) store8<T, L>(kept, begin(k), threads, H, h[k]);
            kept = nullptr;
        }
        const float by = large ? 0x1p-80f : small ? 0x1p100f : 1.f;
        sum = top = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (begin(k) < H)
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    h[k][j] *= by;
                    sum = fmaf(h[k][j], h[k][j], sum);
                }
        if constexpr (!WARP) __syncthreads();  // (the first sums have been read)
        over_row(sum, top);
        inv = rsqrtf(sum / (float)p.H + p.eps * by * by);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (begin(k) < H) {
                float g[kVec];
                load_weight(begin(k), g);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    h[k][j] *= inv;
                    top = max_nan(top, fabsf(h[k][j] * g[j]));
                }
            }
        inv = 1.f;
        if constexpr (kQuant) {
            if constexpr (!WARP) __syncthreads();
            over_row(sum, top);
        }
    }
    // Applied after inv: their product may overflow (a row of zeros). The rounded reciprocal is one
    // rounding more than a division by the scale: 6e-8 of the value, whose code is rounded to 2^-4 of
    // it. Divisions take 171 us for 16384 rows of 8192 instead of 143.
    float per_scale = 1.f;
    if constexpr (kQuant) {
        const float scale = max_nan(inv * top / 448.f, 1.17549435e-38f);
        per_scale = 1.f / scale;
        if (tid == 0) p.out_scale[o] = scale;
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int e = begin(k);
        if (e >= H) continue;
        if (kept) store8<T, L>(kept, e, threads, H, h[k]);
        float g[kVec], y[kVec];
        load_weight(e, g);
#pragma unroll
        for (int j = 0; j < kVec; ++j) y[j] = h[k][j] * inv * g[j] * per_scale;
        if constexpr (kQuant)
            store8_e4m3<L>(reinterpret_cast<uint8_t*>(out), e, threads, H, y);
        else
            store8<O, L>(out, e, threads, H, y);
    }
}

template <typename T, typename O, Layout L, bool WARP, int NV>
__global__ void __launch_bounds__(WARP ? kWarpRows * 32 : (NV == 4 ? 1024 : 512)) k_norm(NormParams p) {
    __shared__ float red[32][2];
    pdl_trigger();
    pdl_wait();
    if constexpr (WARP) {
        const uint32_t o = blockIdx.x * kWarpRows + (threadIdx.x >> 5);
        if (o < p.n) norm_row<T, O, L, true, NV>(p, o, threadIdx.x & 31, 32, nullptr);
    } else {
        norm_row<T, O, L, false, NV>(p, blockIdx.x, threadIdx.x, blockDim.x, red);
    }
}

template <typename T, typename O, bool VEC>
lp_status launch_norm(NormParams p, lp_stream_t s) {
    uint32_t vecs = (p.H + kVec - 1) / kVec;
    if (vecs <= kWarpRowVecs) {
        constexpr Layout L = VEC ? kAligned : kStrided;
        const dim3 grid((p.n + kWarpRows - 1) / kWarpRows);
        if (vecs <= 32) return launch(k_norm<T, O, L, true, 1>, grid, kWarpRows * 32, 0, s, 1, p);
        return launch(k_norm<T, O, L, true, 4>, grid, kWarpRows * 32, 0, s, 1, p);
    }
    constexpr Layout L = VEC ? kAligned : kShifted;
    p.shift = !VEC && vecs < LP_MAX_HIDDEN / kVec;  // (one group more, for which the longest rows have no room)
    if (p.shift) ++vecs;
    const auto warps_for = [&](uint32_t nv) { return ((vecs + nv - 1) / nv + 31) / 32 * 32; };
    // Few rows: as many threads a row as it has vectors (the row's latency counts). Many: fewer
    // threads with more vectors each, so that several rows share an SM and their loads, sums and
    // stores overlap (16384 rows of 8192 bf16 -> e4m3 and residual: 153 us with 512 threads a row,
    // 141 with 256; of 4096: 94 with 512, 75 with 128).
    const bool few = p.n <= 2u * (uint32_t)sm_count();
    if (vecs <= (few ? 512u : 128u)) return launch(k_norm<T, O, L, false, 1>, dim3(p.n), warps_for(1), 0, s, 1, p);
    if (vecs <= (few ? 1024u : 256u)) return launch(k_norm<T, O, L, false, 2>, dim3(p.n), warps_for(2), 0, s, 1, p);
    return launch(k_norm<T, O, L, false, 4>, dim3(p.n), warps_for(4), 0, s, 1, p);
}

template <typename T>
lp_status launch_norm(const NormParams& p, uint32_t out_dtype, uint32_t dtype, bool vec, lp_stream_t s) {
    if (out_dtype == LP_E4M3)
        return vec ? launch_norm<T, uint8_t, true>(p, s) : launch_norm<T, uint8_t, false>(p, s);
    if (out_dtype == dtype) return vec ? launch_norm<T, T, true>(p, s) : launch_norm<T, T, false>(p, s);
    return vec ? launch_norm<T, float, true>(p, s) : launch_norm<T, float, false>(p, s);
}

}  // namespace

extern "C" {

lp_status lp_head_clear_status(void* workspace, lp_stream_t stream) {
    if (!workspace || !aligned_to(workspace, 256)) return LP_ERR_WORKSPACE;
    if (cudaMemsetAsync(workspace, 0, 4, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) {
        (void)cudaGetLastError();
        return LP_ERR_CUDA;
    }
    return LP_OK;
}

lp_status lp_head_norm(const void* x, const void* residual, const void* weight, uint32_t dtype,
                       uint32_t weight_dtype, uint32_t T, uint32_t H, uint64_t x_stride, uint64_t residual_stride,
                       const uint32_t* rows, uint32_t n, float eps, void* out, uint32_t out_dtype,
                       uint64_t out_stride, float* out_scale, void* residual_out, uint64_t residual_out_stride,
                       void* workspace, size_t workspace_bytes, lp_stream_t stream) {
    if (T == 0 || n == 0) return LP_ERR_SHAPE;  // (before the pointers: an empty tensor has none)
    if (!x || !weight || !out) return LP_ERR_NULL;
    if (dtype > LP_F16 || (weight_dtype != dtype && weight_dtype != LP_F32)) return LP_ERR_DTYPE;
    if (out_dtype != dtype && out_dtype != LP_F32 && out_dtype != LP_E4M3) return LP_ERR_DTYPE;
    if (out_dtype == LP_E4M3 && !out_scale) return LP_ERR_NULL;
    if (n > 0x7FFFFFFFu || H == 0 || H > LP_MAX_HIDDEN || (!rows && n != T)) return LP_ERR_SHAPE;
    if (x_stride < H || out_stride < H || (residual && residual_stride < H) ||
        (residual_out && residual_out_stride < H))
        return LP_ERR_SHAPE;
    const size_t e = dtype_bytes(dtype), eo = dtype_bytes(out_dtype), ew = dtype_bytes(weight_dtype);
    if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(residual_out, e) || !aligned_to(weight, ew) ||
        !aligned_to(out, eo) || !aligned_to(out_scale, 4) || !aligned_to(rows, 4))
        return LP_ERR_SHAPE;
    if (!(eps >= 0.f) || eps > 3.0e38f) return LP_ERR_SHAPE;
    if (rows && (!workspace || workspace_bytes < lph::kHeaderBytes)) return LP_ERR_WORKSPACE;
    if (workspace && !aligned_to(workspace, 256)) return LP_ERR_WORKSPACE;
    // An output in an input's place: row for row, so that no row is read after its place was written.
    const auto apart = [&](const void* to, uint32_t type, uint64_t to_stride, const void* from, uint64_t from_stride) {
        return to != from || !to || (!rows && type == dtype && (to_stride == from_stride || T == 1));
    };
    if (!apart(out, out_dtype, out_stride, x, x_stride) || !apart(out, out_dtype, out_stride, residual, residual_stride) ||
        !apart(residual_out, dtype, residual_out_stride, x, x_stride) ||
        !apart(residual_out, dtype, residual_out_stride, residual, residual_stride) || out == residual_out)
        return LP_ERR_SHAPE;
    NormParams p;
    p.x = x;
    p.residual = residual;
    p.weight = weight;
    p.rows = rows;
    p.out = out;
    p.out_scale = out_scale;
    p.residual_out = residual_out;
    p.status = static_cast<uint32_t*>(workspace);
    p.x_stride = x_stride;
    p.residual_stride = residual_stride;
    p.out_stride = out_stride;
    p.residual_out_stride = residual_out_stride;
    p.T = T;
    p.n = n;
    p.H = H;
    p.eps = eps;
    // 16-byte accesses (8 bytes for an e4m3 output) where every row starts on such a boundary
    // and ends on a whole vector; one element at a time otherwise.
    const auto vec_rows = [](const void* ptr, uint64_t stride, size_t size) {
        const size_t bytes = size == 1 ? 8 : 16;
        return !ptr || (lph::aligned_to(ptr, bytes) && stride * size % bytes == 0);
    };
    const bool vec = H % kVec == 0 && vec_rows(x, x_stride, e) && vec_rows(residual, residual_stride, e) &&
                     vec_rows(out, out_stride, eo) && vec_rows(residual_out, residual_out_stride, e) &&
                     aligned_to(weight, 16);
    p.weight_f32 = weight_dtype == LP_F32;
    if (dtype == LP_F32) return launch_norm<float>(p, out_dtype, dtype, vec, stream);
    if (dtype == LP_BF16) return launch_norm<__nv_bfloat16>(p, out_dtype, dtype, vec, stream);
    return launch_norm<__half>(p, out_dtype, dtype, vec, stream);
}

}  // extern "C"
