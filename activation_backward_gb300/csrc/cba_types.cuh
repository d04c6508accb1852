// cba_types.cuh -- element types of the normalisation, attention and
// orthogonalisation operators (cba_dtype_t): conversion to and from fp32,
// vector loads and stores, and the host-side checks they share.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "../../include/cba.h"

namespace cba {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// VEC consecutive elements as they lie in memory; aligned to their size up to
// 16 bytes, so a load or store of one is at most a few 16-byte accesses.
template <typename T, int VEC>
struct __align__(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
    T v[VEC];
};

// Elements 2 j and 2 j + 1 of a pack as fp32, and the other way.
template <typename T, int VEC>
__device__ __forceinline__ float2 pair_of(const Pack<T, VEC> &p, int j) {
    if constexpr (sizeof(T) == 4) {
        return make_float2(p.v[2 * j], p.v[2 * j + 1]);
    } else if constexpr (std::is_same<T, __half>::value) {
        return __half22float2(__halves2half2(p.v[2 * j], p.v[2 * j + 1]));
    } else {
        return __bfloat1622float2(__halves2bfloat162(p.v[2 * j], p.v[2 * j + 1]));
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void set_pair(Pack<T, VEC> &p, int j, float2 v) {
    if constexpr (sizeof(T) == 4) {
        p.v[2 * j] = v.x;
        p.v[2 * j + 1] = v.y;
    } else if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __float22half2_rn(v);
        p.v[2 * j] = h.x;
        p.v[2 * j + 1] = h.y;
    } else {
        const __nv_bfloat162 h = __float22bfloat162_rn(v);
        p.v[2 * j] = h.x;
        p.v[2 * j + 1] = h.y;
    }
}

inline size_t dtype_bytes(int t) { return t == CBA_F32 ? 4 : 2; }
inline bool dtype_ok(int t) { return t == CBA_F32 || t == CBA_F16 || t == CBA_BF16; }
__host__ __device__ inline bool aligned_to(const void *p, size_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Lets a kernel use `bytes` of dynamic shared memory: set once per device (the
// call costs about as much as a launch's arguments).
template <auto Kern>
cudaError_t allow_smem(int bytes) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// The device that holds `ptr` becomes current for this library's runtime
// (cba_api.cu); ordinary host memory is an error.
cudaError_t select_device_of(const void *ptr);

}  // namespace cba
