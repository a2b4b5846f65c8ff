// Element types of the node-update operators: loads widen to fp32, stores round once to nearest.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace uvu {

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }

// V consecutive elements moved as one 16-byte (V > 1) or element-sized (V = 1) access.
template <typename T, int V>
struct Vec {
    static_assert(V == 1 || V * sizeof(T) == 16, "a vector is one element or 16 bytes");
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const T* p) {
    Vec<T, V> r;
    if constexpr (V == 1) {
        r.v[0] = *p;
    } else {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        __builtin_memcpy(&r, &q, 16);
    }
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, V>& r) {
    if constexpr (V == 1) {
        *p = r.v[0];
    } else {
        uint4 q;
        __builtin_memcpy(&q, &r, 16);
        *reinterpret_cast<uint4*>(p) = q;
    }
}

}  // namespace uvu
