// RMS norm of rows of more than 8192 values, which the threads of a block do not hold in registers: see rms.h for the formulas.
//
// A block has a row at a time and goes over it two or three times, each thread over its own columns, so that what it wrote is what it
// reads again: the sum (h is stored), then y; to 8 bits the groups' largest |y| between them, then the values.  The second time the row
// comes from the L2 cache.  The gradient keeps d_gamma's sums of its rows in shared memory, a column a thread.  Bound by the passes, each of
// which waits for the last one's sum and for its own reads: 10,000 x 9216 with the residual in fp32 271 us forward (5.4 TB/s), 280 us back and
// 347 us to 8 bits (3.5 TB/s); in bf16 194, 231 and 281 us.
#include "rms.h"

namespace uvu {
namespace {

constexpr int kWideThreads = 512, kWideBlocks = 4;  // blocks of an SM

__device__ __forceinline__ float block_sum(float v, float* s_part) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();  // the last sums have been read
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kWideThreads / 32; ++w) v += s_part[w];
    return v;
}

// f(column, whether it is inside) for every V columns of this thread, the same number of times in all lanes of a warp.
template <int V, typename F>
__device__ __forceinline__ void each(int width, F f) {
    const int lane = threadIdx.x & 31;
    for (int base = int(threadIdx.x - lane) * V; base < width; base += kWideThreads * V) f(base + lane * V, base + lane * V < width);
}
template <typename T, int V>
__device__ __forceinline__ void read(const T* p, float (&v)[V]) {
    const Pack<T, V> q = *reinterpret_cast<const Pack<T, V>*>(p);
    q.get(v);
}
template <typename T, int V>
__device__ __forceinline__ void write(T* p, const float (&v)[V]) {
    Pack<T, V> o;
    o.set(v);
    *reinterpret_cast<Pack<T, V>*>(p) = o;
}
// gamma of columns c .. c + V - 1
template <int V>
__device__ __forceinline__ void gammas(const RmsArgs& a, int c, float (&g)[V]) {
    int ch = c / a.inner, i = c - ch * a.inner;
    if (a.inner >= V) {  // of two channels at most
        const int left = a.inner - i;
        const float first = a.gamma[ch], second = left < V ? a.gamma[ch + 1] : 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) g[k] = k < left ? first : second;
        return;
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
        g[k] = a.gamma[ch];
        if (++i == a.inner) i = 0, ++ch;
    }
}

template <typename T, int V, RmsMode MODE>
__global__ void __launch_bounds__(kWideThreads) rms_wide_kernel(const RmsArgs a) {
    static_assert(MODE == kRmsFwd || MODE == kRmsQuant);
    __shared__ float s_part[kWideThreads / 32];
    extern __shared__ unsigned s_top[];  // [groups]
    const float inv = 1.f / float(a.width);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t at = row * a.width;
        const T* x = static_cast<const T*>(a.in[0]) + at;
        const T* res = a.in[1] ? static_cast<const T*>(a.in[1]) + at : nullptr;
        T* h = static_cast<T*>(a.out[1]) + (res ? at : 0);
        const T* stored = res ? h : x;
        float s = 0.f;
        each<V>(a.width, [&](int c, bool inside) {
            if (!inside) return;
            float v[V];
            read<T, V>(x + c, v);
            if (res) {
                float u[V];
                read<T, V>(res + c, u);
#pragma unroll
                for (int i = 0; i < V; ++i) u[i] += v[i];
                Pack<T, V> o;
                o.set(u);
                o.get(v);
                *reinterpret_cast<Pack<T, V>*>(h + c) = o;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) s = fmaf(v[i], v[i], s);
        });
        const float mean = fmaf(block_sum(s, s_part), inv, a.eps);
        float r = inv_sqrt(mean);
        if (squares_beyond(mean)) {
            const float f = squares_factor(mean);
            s = 0.f;
            each<V>(a.width, [&](int c, bool inside) {
                if (!inside) return;
                float v[V];
                read<T, V>(stored + c, v);
#pragma unroll
                for (int i = 0; i < V; ++i) s = fmaf(v[i] * f, v[i] * f, s);
            });
            r = inv_sqrt(fmaf(block_sum(s, s_part), inv, a.eps * f * f)) * f;
        }
        auto normal = [&](int c, float (&v)[V]) {
            float g[V];
            read<T, V>(stored + c, v);
            gammas<V>(a, c, g);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = v[i] * r * g[i];
        };
        if constexpr (MODE == kRmsFwd) {
            if (a.rstd && threadIdx.x == 0) a.rstd[row] = r;
            T* y = static_cast<T*>(a.out[0]) + at;
            each<V>(a.width, [&](int c, bool inside) {
                if (!inside) return;
                float v[V];
                normal(c, v);
                write<T, V>(y + c, v);
            });
        } else {
            for (int j = threadIdx.x; j < a.groups; j += kWideThreads) s_top[j] = 0u;  // the last row's have been read: block_sum
            __syncthreads();
            const bool by_warp = a.groups == 1 || a.group % (32 * V) == 0;  // the lanes of a step share a group
            each<V>(a.width, [&](int c, bool inside) {
                float v[V] = {}, top = 0.f;
                if (inside) normal(c, v);
#pragma unroll
                for (int i = 0; i < V; ++i) top = nan_max(top, fabsf(v[i]));
                const int g = c / a.group;
                if (by_warp) {
                    const unsigned most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
                    if ((threadIdx.x & 31) == 0) atomicMax(s_top + g, most);
                } else if (inside) {
                    if ((c + V - 1) / a.group == g) {
                        atomicMax(s_top + g, __float_as_uint(top));
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) atomicMax(s_top + (c + i) / a.group, __float_as_uint(fabsf(v[i])));
                    }
                }
            });
            __syncthreads();
            uint8_t* q = static_cast<uint8_t*>(a.out[0]) + at;
            auto divide = [&](int g, const float* v, auto& u) {
                const Scale scale(__uint_as_float(s_top[g]));
                if (__builtin_expect(scale.rare(), 0)) scale.template divide<true>(v, u);
                else scale.template divide<false>(v, u);
            };
            each<V>(a.width, [&](int c, bool inside) {
                if (!inside) return;
                float v[V], u[V];
                normal(c, v);
                const int g = c / a.group;
                if ((c + V - 1) / a.group == g) {
                    divide(g, v, u);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float one[1];
                        divide((c + i) / a.group, v + i, one);
                        u[i] = one[0];
                    }
                }
                Bytes<V> o;
                o.set(u);
                *reinterpret_cast<Bytes<V>*>(q + c) = o;
            });
            for (int j = threadIdx.x; j < a.groups; j += kWideThreads) a.scales[row * a.groups + j] = Scale(__uint_as_float(s_top[j])).s;
        }
    }
}

// Rows block_rows b .. of block b, and its sums of d_gamma.
template <typename T, int V>
__global__ void __launch_bounds__(kWideThreads) rms_wide_bwd_kernel(const RmsArgs a) {
    __shared__ float s_part[kWideThreads / 32];
    extern __shared__ __align__(128) float s_sum[];  // [width]: of d_y u, by the thread that has the column
    const float inv = 1.f / float(a.width);
    const T *H = static_cast<const T*>(a.in[0]), *DY = static_cast<const T*>(a.in[1]), *DH = static_cast<const T*>(a.in[2]);
    T* DX = static_cast<T*>(a.out[0]);
    each<V>(a.width, [&](int c, bool inside) {
        const float none[V] = {};
        if (inside) write<float, V>(s_sum + c, none);
    });
    const int64_t first = int64_t(blockIdx.x) * a.block_rows, end = min(first + a.block_rows, a.rows);
    for (int64_t row = first; row < end; ++row) {
        const int64_t at = row * a.width;
        const float r = a.rstd[row];
        float dot = 0.f;
        each<V>(a.width, [&](int c, bool inside) {
            if (!inside) return;
            float x[V], g[V], gamma[V], sum[V];
            read<T, V>(H + at + c, x);
            read<T, V>(DY + at + c, g);
            read<float, V>(s_sum + c, sum);
            gammas<V>(a, c, gamma);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float u = x[i] * r;
                sum[i] = fmaf(g[i], u, sum[i]);
                dot = fmaf(g[i] * gamma[i], u, dot);
            }
            write<float, V>(s_sum + c, sum);
        });
        const float mean = block_sum(dot, s_part) * inv;  // of t u
        each<V>(a.width, [&](int c, bool inside) {
            if (!inside) return;
            float x[V], g[V], t[V] = {}, gamma[V];
            read<T, V>(H + at + c, x);
            read<T, V>(DY + at + c, g);
            if (DH) read<T, V>(DH + at + c, t);
            gammas<V>(a, c, gamma);
#pragma unroll
            for (int i = 0; i < V; ++i) t[i] = fmaf(fmaf(-x[i] * r, mean, g[i] * gamma[i]), r, t[i]);
            write<T, V>(DX + at + c, t);
        });
    }
    __syncthreads();
    const int channels = a.width / a.inner, lane = threadIdx.x & 31;
    for (int c = threadIdx.x >> 5; c < channels; c += kWideThreads / 32) {  // a warp for each: there may be one channel of all components
        float s = 0.f;
        for (int i = lane; i < a.inner; i += 32) s += s_sum[c * a.inner + i];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == 0) a.partial[int64_t(blockIdx.x) * channels + c] = s;
    }
}

// f(V): vectors of 16 bytes where every row of every tensor begins on one (an 8-bit one: on V bytes), else single values.
template <typename T, typename F>
cudaError_t by_alignment(const RmsArgs& a, bool quant, F f) {
    uintptr_t any = uintptr_t(a.width) * sizeof(T) | reinterpret_cast<uintptr_t>(a.out[0]) * (quant ? sizeof(T) : 1);
    any |= reinterpret_cast<uintptr_t>(a.out[1]);
    for (const void* t : a.in) any |= reinterpret_cast<uintptr_t>(t);
    return any % 16 == 0 ? f(std::integral_constant<int, 16 / int(sizeof(T))>()) : f(std::integral_constant<int, 1>());
}

template <typename T>
cudaError_t wide_launch(const RmsArgs& a, RmsMode mode, int sms, cudaStream_t st) {
    return by_alignment<T>(a, mode == kRmsQuant, [&](auto v) {
        constexpr int V = decltype(v)::value;
        auto kernel = mode == kRmsFwd     ? rms_wide_kernel<T, V, kRmsFwd>
                      : mode == kRmsQuant ? rms_wide_kernel<T, V, kRmsQuant>
                                          : rms_wide_bwd_kernel<T, V>;
        const size_t smem = mode == kRmsFwd ? 0 : size_t(mode == kRmsQuant ? a.groups : a.width) * 4;
        if (smem > 40 << 10) {
            cudaError_t e = allow_most_smem(kernel, smem);
            if (e != cudaSuccess) return e;
        }
        const int64_t blocks = mode == kRmsBwd ? (a.rows + a.block_rows - 1) / a.block_rows : std::min<int64_t>(a.rows, int64_t(sms) * kWideBlocks);
        kernel<<<unsigned(blocks), kWideThreads, smem, st>>>(a);
        return cudaGetLastError();
    });
}

}  // namespace

int64_t rms_wide_blocks(int64_t rows, int sms) { return std::min(rows, std::max(int64_t(sms) * kWideBlocks, (rows + kTeamRows - 1) / kTeamRows)); }

namespace {
cudaError_t launch(uvu_dtype dtype, const RmsArgs& a, RmsMode mode, int sms, cudaStream_t st) {
    switch (dtype) {
        case UVU_F32: return wide_launch<float>(a, mode, sms, st);
        case UVU_BF16: return wide_launch<__nv_bfloat16>(a, mode, sms, st);
        case UVU_F16: return wide_launch<__half>(a, mode, sms, st);
        default: return cudaErrorInvalidValue;
    }
}
}  // namespace

cudaError_t launch_rms_wide_fwd(const RmsShape& s, const void* x, const void* residual, const float* gamma, void* h, void* y, float* rstd,
                                int sms, cudaStream_t st) {
    return launch(s.dtype, rms_fwd_args(s, x, residual, gamma, h, y, rstd), kRmsFwd, sms, st);
}
cudaError_t launch_rms_wide_quant(const RmsShape& s, int group, const void* x, const void* residual, const float* gamma, void* h, void* q,
                                  float* scales, int sms, cudaStream_t st) {
    return launch(s.dtype, rms_quant_args(s, group, x, residual, gamma, h, q, scales), kRmsQuant, sms, st);
}
cudaError_t launch_rms_wide_bwd(const RmsShape& s, const void* dy, const void* h, const float* gamma, const float* rstd, const void* dh,
                                void* dx, float* partial, int sms, cudaStream_t st, int64_t* blocks) {
    RmsArgs a = rms_bwd_args(s, dy, h, gamma, rstd, dh, dx, partial);
    const int64_t most = rms_wide_blocks(a.rows, sms);
    a.block_rows = (a.rows + most - 1) / most;
    *blocks = (a.rows + a.block_rows - 1) / a.block_rows;
    return launch(s.dtype, a, kRmsBwd, sms, st);
}

}  // namespace uvu
