// Root-mean-square norm with the residual's addition, its gradient, and the form with 8-bit output.
//
//     h = round(x + residual),  r = (mean h^2 + eps)^(-1/2),  y = h r gamma          (a row: channels * inner values)
//     8 bits, for each group of a row:  s = max |y| / 448,  q = e4m3(y / s)
//     d_x = d_h + r (t - u mean(t u)),  t = gamma d_y,  u = h r;   d_gamma[c] = sum over rows and components of d_y u
//
// gamma is one value a channel, shared by the `inner` components of an irrep, so y is as equivariant as x.  The norm is of h as
// it is stored: what the next layer and the gradient read is what was normalised.
//
// Bound by memory: every tensor moves once.  A row belongs to a team, a part of a warp or a block, whose threads hold the row in
// registers between the sum and the result; a thread has the same columns of every row that it sees, so gamma is read once
// and d_gamma is summed in registers, then over the block's teams in shared memory, and over the blocks, in their order, by a
// second kernel.
#include <cuda_fp8.h>

#include <algorithm>
#include <cstdint>

#include "elem.h"
#include "plan.h"

namespace uvu {
namespace {

constexpr float kTop = 448.f;  // the largest e4m3 value
constexpr int kRunRows = 512;  // rows that a team adds up in one fp32 sum of d_gamma

// Columns of a thread: vector k of the row's vectors lane, lane + team, ...
struct Team {
    int row0, rows, lane, size;  // row of this thread in a step, rows of a step (over the grid), thread of the team
};

// Sum over the team, in every thread of it.  WARP: team is a power of two of lanes.
template <bool WARP>
__device__ __forceinline__ float team_sum(float v, int size, float* s_part) {
    if (WARP) {
        for (int d = size >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        return v;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    const int warps = size >> 5;
    __syncthreads();  // the last sum has been read
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < warps; ++w) v += s_part[w];
    return v;
}

template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, V>& r) {
    *reinterpret_cast<Pack<T, V>*>(p) = r;
}

struct RmsArgs {
    int64_t rows;
    int width, inner, team, group, groups;  // width: values of a row; group: values that share a scale
    float eps;
    const void *x, *residual, *dh;
    const float* gamma;
    void *h, *y;
    float *rstd, *scales, *partial;
};

template <typename T, int V, int K, bool WARP, bool QUANT>
__global__ void __launch_bounds__(WARP ? 256 : 512) rms_fwd_kernel(const RmsArgs a) {
    __shared__ float s_part[16];
    extern __shared__ unsigned s_top[];  // largest |y| of each group, for each team of the block
    const int team = WARP ? a.team : blockDim.x, lane = WARP ? threadIdx.x & (team - 1) : threadIdx.x;
    const int per_block = WARP ? blockDim.x / team : 1;
    const int mine = WARP ? threadIdx.x / team : 0;
    const T *x = static_cast<const T*>(a.x), *res = static_cast<const T*>(a.residual);
    T* h = static_cast<T*>(a.h);
    float gamma[K * V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = (k * team + lane) * V + i;
            gamma[k * V + i] = e < a.width ? a.gamma[e / a.inner] : 0.f;
        }
    const float inv = 1.f / float(a.width);
    for (int64_t base = int64_t(blockIdx.x) * per_block; base < a.rows; base += int64_t(gridDim.x) * per_block) {
        const int64_t row = base + mine;
        const bool live = row < a.rows;
        const int64_t at = row * a.width;
        Pack<T, V> xv[K], rv[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = (k * team + lane) * V;
            if (live && e < a.width) {
                xv[k] = load_pack<T, V>(x + at + e);
                if (res) rv[k] = load_pack<T, V>(res + at + e);
            }
        }
        float v[K * V], sum = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = (k * team + lane) * V;
            const bool on = live && e < a.width;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float t = on ? widen(xv[k].v[i]) : 0.f;
                if (res && on) {
                    xv[k].v[i] = narrow<T>(t + widen(rv[k].v[i]));
                    t = widen(xv[k].v[i]);
                }
                v[k * V + i] = t;
                sum = fmaf(t, t, sum);
            }
            if (res && on) store_pack<T, V>(h + at + e, xv[k]);
        }
        sum = team_sum<WARP>(sum, team, s_part);
        const float r = 1.f / sqrtf(sum * inv + a.eps);
        if (live && lane == 0 && a.rstd) a.rstd[row] = r;
        if (!QUANT) {
            T* y = static_cast<T*>(a.y);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int e = (k * team + lane) * V;
                if (live && e < a.width) {
                    Pack<T, V> o;
#pragma unroll
                    for (int i = 0; i < V; ++i) o.v[i] = narrow<T>(v[k * V + i] * r * gamma[k * V + i]);
                    store_pack<T, V>(y + at + e, o);
                }
            }
        } else {
            unsigned* top = s_top + mine * a.groups;
            if (WARP) __syncwarp(); else __syncthreads();  // the last row's maxima have been read
            for (int j = lane; j < a.groups; j += team) top[j] = 0u;
            if (WARP) __syncwarp(); else __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int e = (k * team + lane) * V;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[k * V + i] *= r * gamma[k * V + i];
                    if (live && e < a.width) atomicMax(top + (e + i) / a.group, __float_as_uint(fabsf(v[k * V + i])));
                }
            }
            if (WARP) __syncwarp(); else __syncthreads();
            __nv_fp8_e4m3* y = static_cast<__nv_fp8_e4m3*>(a.y);
            if (live) {
                for (int j = lane; j < a.groups; j += team) a.scales[row * a.groups + j] = __uint_as_float(top[j]) / kTop;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int e = (k * team + lane) * V;
                    if (e < a.width) {
                        Pack<__nv_fp8_e4m3, V> o;
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float s = __uint_as_float(top[(e + i) / a.group]) / kTop;
                            o.v[i] = __nv_fp8_e4m3(s == 0.f ? 0.f : v[k * V + i] / s);
                        }
                        store_pack<__nv_fp8_e4m3, V>(y + at + e, o);
                    }
                }
            }
        }
    }
}

// x is h here.  partial [gridDim.x][channels]
template <typename T, int V, int K, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 512) rms_bwd_kernel(const RmsArgs a, const void* dyp, int64_t block_rows) {
    __shared__ float s_part[16];
    extern __shared__ float s_sum[];  // [width]
    const int team = WARP ? a.team : blockDim.x, lane = WARP ? threadIdx.x & (team - 1) : threadIdx.x;
    const int per_block = WARP ? blockDim.x / team : 1;
    const int mine = WARP ? threadIdx.x / team : 0;
    const T *x = static_cast<const T*>(a.x), *dy = static_cast<const T*>(dyp), *dh = static_cast<const T*>(a.dh);
    T* dx = static_cast<T*>(a.y);
    float gamma[K * V], acc[K * V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = (k * team + lane) * V + i;
            gamma[k * V + i] = e < a.width ? a.gamma[e / a.inner] : 0.f;
            acc[k * V + i] = 0.f;
        }
    const float inv = 1.f / float(a.width);
    const int64_t first = int64_t(blockIdx.x) * block_rows, end = min(first + block_rows, a.rows);
    for (int64_t base = first; base < end; base += per_block) {
        const int64_t row = base + mine;
        const bool live = row < end;
        const int64_t at = row * a.width;
        Pack<T, V> xv[K], gv[K], hv[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = (k * team + lane) * V;
            if (live && e < a.width) {
                xv[k] = load_pack<T, V>(x + at + e);
                gv[k] = load_pack<T, V>(dy + at + e);
                if (dh) hv[k] = load_pack<T, V>(dh + at + e);
            }
        }
        const float r = live ? a.rstd[row] : 0.f;
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = (k * team + lane) * V;
            if (live && e < a.width) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float u = widen(xv[k].v[i]) * r, g = widen(gv[k].v[i]);
                    acc[k * V + i] = fmaf(g, u, acc[k * V + i]);
                    dot = fmaf(g * gamma[k * V + i], u, dot);
                }
            }
        }
        dot = team_sum<WARP>(dot, team, s_part) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int e = (k * team + lane) * V;
            if (live && e < a.width) {
                Pack<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float u = widen(xv[k].v[i]) * r;
                    float t = r * fmaf(widen(gv[k].v[i]), gamma[k * V + i], -u * dot);
                    if (dh) t += widen(hv[k].v[i]);
                    o.v[i] = narrow<T>(t);
                }
                store_pack<T, V>(dx + at + e, o);
            }
        }
    }
    // over the block's teams, in their order, then over a channel's components
    for (int m = 0; m < per_block; ++m) {
        if (mine == m) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int e = (k * team + lane) * V + i;
                    if (e < a.width) s_sum[e] = m == 0 ? acc[k * V + i] : s_sum[e] + acc[k * V + i];
                }
        }
        __syncthreads();
    }
    const int channels = a.width / a.inner;
    for (int c = threadIdx.x; c < channels; c += blockDim.x) {
        float s = 0.f;
        for (int i = 0; i < a.inner; ++i) s += s_sum[c * a.inner + i];
        a.partial[int64_t(blockIdx.x) * channels + c] = s;
    }
}

// d_gamma[c] = sum over the blocks of partial[b][c]: 32 channels a block, 32 threads for each.
__global__ void __launch_bounds__(1024) rms_join_kernel(const float* partial, int blocks, int channels, float* out) {
    __shared__ float s[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float sum = 0.f;
    if (c < channels)
        for (int b = threadIdx.y; b < blocks; b += 32) sum += partial[int64_t(b) * channels + c];
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    sum = s[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const int out_c = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && out_c < channels) out[out_c] = sum;
}

struct RmsPlan {
    bool warp;
    int v, k, team, threads;
};
// Vectors of 16 bytes where every row of every tensor begins on one, else of 4 bytes (two 16-bit values) or single values.  A team
// of up to a warp while its threads hold at most 32 values, a block beyond.
RmsPlan rms_plan(int width, int size, uintptr_t any) {
    RmsPlan p;
    const uintptr_t row = uintptr_t(width) * size | any;
    p.v = row % 16 == 0 ? 16 / size : row % 4 == 0 ? 4 / size : 1;
    const int vecs = (width + p.v - 1) / p.v;
    p.warp = width <= 1024;
    if (p.warp) {
        p.team = 1;
        while (p.team < 32 && p.team < vecs) p.team *= 2;
        p.k = 1;
        while (p.k * p.team < vecs) p.k *= 2;
        p.threads = 256;
    } else {
        p.k = 16 / p.v;
        p.threads = p.team = std::min(512, ((vecs + p.k - 1) / p.k + 31) / 32 * 32);
    }
    return p;
}

template <typename F>
cudaError_t by_shape(const RmsPlan& p, int size, F f) {
    auto at = [&](auto v, auto k) -> cudaError_t { return p.warp ? f(v, k, std::true_type()) : f(v, k, std::false_type()); };
    auto I = [](auto n) { return n; };
    (void)I;
#define UVU_AT(V_, K_) \
    if (p.v == V_ && p.k == K_) return at(std::integral_constant<int, V_>(), std::integral_constant<int, K_>());
    if (size == 4) {
        UVU_AT(4, 1) UVU_AT(4, 2) UVU_AT(4, 4) UVU_AT(4, 8)
    } else {
        UVU_AT(8, 1) UVU_AT(8, 2) UVU_AT(8, 4) UVU_AT(2, 1) UVU_AT(2, 2) UVU_AT(2, 4) UVU_AT(2, 8) UVU_AT(2, 16)
    }
    UVU_AT(1, 1) UVU_AT(1, 2) UVU_AT(1, 4) UVU_AT(1, 8) UVU_AT(1, 16) UVU_AT(1, 32)
#undef UVU_AT
    return cudaErrorInvalidValue;
}

int64_t bwd_block_rows(const RmsPlan& p, int64_t rows, int sms) {
    const int64_t teams = p.warp ? p.threads / p.team : 1;
    const int64_t blocks = int64_t(sms) * (p.warp ? 4 : 2);
    const int64_t even = ((rows + blocks - 1) / blocks + teams - 1) / teams * teams;
    return std::min<int64_t>(even, kRunRows * teams);
}

template <typename T>
cudaError_t fwd(const RmsShape& s, RmsArgs a, bool quant, int sms, cudaStream_t st) {
    const uintptr_t any = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual) | reinterpret_cast<uintptr_t>(a.h) |
                          (quant ? reinterpret_cast<uintptr_t>(a.y) * sizeof(T) : reinterpret_cast<uintptr_t>(a.y));
    const RmsPlan p = rms_plan(a.width, sizeof(T), any);
    a.team = p.team;
    const int64_t teams = p.warp ? p.threads / p.team : 1;
    const unsigned grid = unsigned(std::min<int64_t>((s.rows + teams - 1) / teams, int64_t(sms) * 8));
    const size_t smem = quant ? size_t(teams) * a.groups * 4 : 0;
    return by_shape(p, sizeof(T), [&](auto v, auto k, auto warp) {
        constexpr int V = decltype(v)::value, K = decltype(k)::value;
        constexpr bool W = decltype(warp)::value;
        if constexpr (V * sizeof(T) <= 16 && V * K <= 32) {
            if (quant)
                rms_fwd_kernel<T, V, K, W, true><<<grid, p.threads, smem, st>>>(a);
            else
                rms_fwd_kernel<T, V, K, W, false><<<grid, p.threads, 0, st>>>(a);
            return cudaGetLastError();
        }
        return cudaErrorInvalidValue;
    });
}

template <typename T>
cudaError_t bwd(const RmsShape& s, RmsArgs a, const void* dy, float* dgamma, int sms, cudaStream_t st) {
    const uintptr_t any = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.dh) | reinterpret_cast<uintptr_t>(a.y) |
                          reinterpret_cast<uintptr_t>(dy);
    const RmsPlan p = rms_plan(a.width, sizeof(T), any);
    a.team = p.team;
    const int64_t each = bwd_block_rows(p, s.rows, sms), blocks = (s.rows + each - 1) / each;
    cudaError_t e = by_shape(p, sizeof(T), [&](auto v, auto k, auto warp) {
        constexpr int V = decltype(v)::value, K = decltype(k)::value;
        constexpr bool W = decltype(warp)::value;
        if constexpr (V * sizeof(T) <= 16 && V * K <= 32) {
            rms_bwd_kernel<T, V, K, W><<<unsigned(blocks), p.threads, size_t(a.width) * 4, st>>>(a, dy, each);
            return cudaGetLastError();
        }
        return cudaErrorInvalidValue;
    });
    if (e != cudaSuccess) return e;
    rms_join_kernel<<<(s.channels + 31) / 32, dim3(32, 32), 0, st>>>(a.partial, int(blocks), s.channels, dgamma);
    return cudaGetLastError();
}

RmsArgs args_of(const RmsShape& s) {
    RmsArgs a = {};
    a.rows = s.rows;
    a.width = s.channels * s.inner;
    a.inner = s.inner;
    a.eps = float(s.eps);
    return a;
}

}  // namespace

size_t rms_workspace(const RmsShape& s, int sms) {
    if (s.rows == 0) return 0;
    // the alignment of the tensors is not known here: the most blocks of any
    int64_t most = 0;
    const int width = s.channels * s.inner, size = s.dtype == UVU_F32 ? 4 : 2;
    for (uintptr_t any : {0, 4, 2, 1}) {
        const int64_t each = bwd_block_rows(rms_plan(width, size, any), s.rows, sms);
        most = std::max(most, (s.rows + each - 1) / each);
    }
    return size_t(most) * s.channels * 4;
}

cudaError_t launch_rms_fwd(const RmsShape& s, const void* x, const void* residual, const float* gamma, void* h, void* y, float* rstd,
                           int sms, cudaStream_t st) {
    RmsArgs a = args_of(s);
    a.x = x, a.residual = residual, a.gamma = gamma, a.h = h, a.y = y, a.rstd = rstd;
    switch (s.dtype) {
        case UVU_F32: return fwd<float>(s, a, false, sms, st);
        case UVU_BF16: return fwd<__nv_bfloat16>(s, a, false, sms, st);
        case UVU_F16: return fwd<__half>(s, a, false, sms, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_rms_quant(const RmsShape& s, int group, const void* x, const void* residual, const float* gamma, void* h, void* q,
                             float* scales, int sms, cudaStream_t st) {
    RmsArgs a = args_of(s);
    a.x = x, a.residual = residual, a.gamma = gamma, a.h = h, a.y = q, a.scales = scales;
    a.group = group ? group : a.width;
    a.groups = (a.width + a.group - 1) / a.group;
    switch (s.dtype) {
        case UVU_F32: return fwd<float>(s, a, true, sms, st);
        case UVU_BF16: return fwd<__nv_bfloat16>(s, a, true, sms, st);
        case UVU_F16: return fwd<__half>(s, a, true, sms, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_rms_bwd(const RmsShape& s, const void* dy, const void* h, const float* gamma, const float* rstd, const void* dh,
                           void* dx, float* dgamma, void* ws, int sms, cudaStream_t st) {
    if (s.rows == 0) return cudaMemsetAsync(dgamma, 0, size_t(s.channels) * 4, st);
    RmsArgs a = args_of(s);
    a.x = h, a.gamma = gamma, a.dh = dh, a.y = dx, a.rstd = const_cast<float*>(rstd), a.partial = static_cast<float*>(ws);
    switch (s.dtype) {
        case UVU_F32: return bwd<float>(s, a, dy, dgamma, sms, st);
        case UVU_BF16: return bwd<__nv_bfloat16>(s, a, dy, dgamma, sms, st);
        case UVU_F16: return bwd<__half>(s, a, dy, dgamma, sms, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace uvu
