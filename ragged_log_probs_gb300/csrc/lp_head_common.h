// Shared pieces of the head operators' kernels (final norm, projection, logits processing).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "lp_head.h"

namespace lph {

constexpr size_t kHeaderBytes = 256;  // the status word is the header's first word

// Programmatic dependent launch: let the next kernel on the stream start launching, and
// wait until the previous one has finished and its writes are visible. A call's first kernel
// waits before it touches global memory, and where the call has a second one it triggers only
// after that wait. So the second kernel may read the call's inputs, and set status bits, before
// its own wait: what came before the call is complete then. What the first kernel writes, and
// the call's outputs, are touched after it.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void flag(uint32_t* status, uint32_t code) {
    if (status) atomicOr(status, 1u << code);
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN when either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two packed 16-bit values -> two floats.
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// The request of row t: the b with off[b] <= t < off[b+1], or -1. The row's own number is tried
// first (a request a row). Ends for any contents of off (the interval halves each time).
__device__ __forceinline__ int request_of(const uint32_t* off, uint32_t B, uint32_t t) {
    if (!off) return (int)t;
    uint32_t lo = 0, hi = B;  // off[lo] <= t is kept, off[hi] > t is kept, once checked below
    const uint32_t guess = t < B ? t : B - 1, at = off[guess], after = off[guess + 1], begin = off[0], end = off[B];
    if (at <= t && t < after) return (int)guess;
    if (begin > t || end <= t) return -1;
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (off[mid] <= t) lo = mid; else hi = mid;
    }
    return (int)lo;
}

inline size_t dtype_bytes(uint32_t d) { return d == LP_F32 ? 4 : d == LP_E4M3 ? 1 : 2; }
inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int kMaxDevices = 64;

inline int current_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)cudaGetLastError();
        return -1;
    }
    return dev;
}

// SMs of the current device, asked once per device; 0 on failure.
inline int sm_count() {
    static std::atomic<int> known[kMaxDevices];
    const int dev = current_device();
    if (dev < 0) return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
            (void)cudaGetLastError();
            return 0;
        }
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Allow `kernel` that much dynamic shared memory on the current device (once: `set` has a
// bit for each device).
inline bool allow_smem(const void* kernel, size_t bytes, std::atomic<uint64_t>* set) {
    const int dev = current_device();
    if (dev < 0) return false;
    const uint64_t bit = 1ull << dev;
    if (set->load(std::memory_order_acquire) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    set->fetch_or(bit, std::memory_order_release);
    return true;
}

// Launch on `stream` as a programmatic dependent of the previous kernel (cluster > 1: in
// thread-block clusters of that many CTAs along x).
template <typename... Params, typename... Args>
lp_status launch(void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem, lp_stream_t stream,
                 unsigned cluster, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...) != cudaSuccess) {
        (void)cudaGetLastError();
        return LP_ERR_CUDA;
    }
    return LP_OK;
}

}  // namespace lph
