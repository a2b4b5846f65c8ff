// Element types of the node-update operators: loads widen to fp32, stores round once to nearest.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

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

// Two values rounded to 16 bits, `lo` in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// V consecutive values as they lie in memory, taken apart and put together two at a time: with one conversion a value the RMS norm
// was bound by its 39 instructions a value (forward in bf16).
// WORDS: 16-bit values are held as words.  As values they are loaded and cleared one by one where a condition stands before the load.
template <typename T, int V, bool WORDS = true>
struct alignas(V * sizeof(T)) Pack {
    static constexpr bool kPairs = WORDS && sizeof(T) == 2 && V % 2 == 0;
    static constexpr int kEach = kPairs ? 2 : 1;
    using Held = std::conditional_t<kPairs, uint32_t, T>;
    Held t[V / kEach];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < V / kEach; ++i) t[i] = Held(0.f);
    }
    // Value i (known when compiled) of a pack that has been cleared, or all of whose others are there.
    __device__ __forceinline__ void put(int i, T v) {
        if constexpr (kPairs) {
            uint16_t bits;
            __builtin_memcpy(&bits, &v, 2);
            t[i / 2] = __byte_perm(t[i / 2], bits, i % 2 ? 0x5410 : 0x3254);
        } else {
            t[i] = v;
        }
    }
    __device__ __forceinline__ void get(float* v) const {
        if constexpr (sizeof(T) == 4 || V == 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = widen(t[i]);
        } else {
            uint32_t w[(V + 1) / 2];
            __builtin_memcpy(w, t, sizeof(w));
#pragma unroll
            for (int i = 0; i < (V + 1) / 2; ++i) {
                if constexpr (__is_same(T, __nv_bfloat16)) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                    v[2 * i] = f.x, v[2 * i + 1] = f.y;
                }
            }
        }
    }
    __device__ __forceinline__ void set(const float* v) {
        if constexpr (sizeof(T) == 4 || V == 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] = narrow<T>(v[i]);
        } else {
            uint32_t w[(V + 1) / 2];
#pragma unroll
            for (int i = 0; i < (V + 1) / 2; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
            __builtin_memcpy(t, w, sizeof(w));
        }
    }
};
// Pairs of fp32 values: one packed instruction does both (add, mul, fma .f32x2), which halves the
// arithmetic that a value costs beside its special-function instructions.
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
    __device__ __forceinline__ float2 both() const {
        float2 r;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
        return r;
    }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

}  // namespace uvu
