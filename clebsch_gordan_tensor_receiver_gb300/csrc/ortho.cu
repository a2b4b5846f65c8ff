// Orthogonalised updates by Newton-Schulz products.
//
//     X_0 = G / (|G|_F + eps),   P = X X^T,   X <- a X + (b P + c P P) X,   out = scale X after `steps` of them
//
// on the side of the smaller Gram matrix (a tall G is turned).
#include <algorithm>
#include <cstdint>

#include "elem.h"
#include "plan.h"

namespace uvu {
namespace {

// |G|_F in fp32 for values of any size: squares of large and of small values are summed at scales of their own.
template <typename T>
__global__ void __launch_bounds__(512) norm_kernel(int rows, int cols, int64_t g_matrix, int64_t g_row, float eps, const T* g, float* inv) {
    const T* a = g + int64_t(blockIdx.x) * g_matrix;
    float sum[3] = {0.f, 0.f, 0.f};
    const float up = 0x1p60f, down = 0x1p-60f;
    for (int64_t i = threadIdx.x; i < int64_t(rows) * cols; i += blockDim.x) {
        const int64_t r = i / cols;
        const float v = fabsf(widen(a[r * g_row + (i - r * cols)]));
        const int k = v > 0x1p50f ? 2 : v < 0x1p-50f ? 0 : 1;
        const float t = k == 2 ? v * down : k == 0 ? v * up : v;
        sum[k] = fmaf(t, t, sum[k]);
    }
    __shared__ double s[16];
    double total = double(sum[0]) * 0x1p-120 + double(sum[1]) + double(sum[2]) * 0x1p120;
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        total = 0;
        for (int w = 0; w < 16; ++w) total += s[w];
        inv[blockIdx.x] = float(1.0 / (sqrt(total) + double(eps)));
    }
}

template <typename T>
__global__ void take_kernel(int m, int n, bool turned, int64_t g_matrix, int64_t g_row, const T* g, const float* inv, float* x) {
    const int64_t per = int64_t(m) * n;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < per; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t r = i / n, c = i - r * n;
        const T* a = g + int64_t(blockIdx.y) * g_matrix;
        x[int64_t(blockIdx.y) * per + i] = widen(turned ? a[c * g_row + r] : a[r * g_row + c]) * inv[blockIdx.y];
    }
}

template <typename T>
__global__ void give_kernel(int m, int n, bool turned, int64_t o_matrix, int64_t o_row, float scale, const float* x, T* out) {
    const int64_t per = int64_t(m) * n;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < per; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t r = i / n, c = i - r * n;
        T* o = out + int64_t(blockIdx.y) * o_matrix;
        o[turned ? c * o_row + r : r * o_row + c] = narrow<T>(x[int64_t(blockIdx.y) * per + i] * scale);
    }
}

// C [m][n] = alpha op(A B) + beta D: A [m][k], B [k][n] or (TB) [n][k]; D like C.
template <bool TB>
__global__ void __launch_bounds__(256) product_kernel(int m, int n, int k, const float* A, const float* B, float alpha, const float* D,
                                                      float beta, float* C) {
    __shared__ float sa[16][65], sb[16][65];
    A += int64_t(blockIdx.z) * m * k;
    B += int64_t(blockIdx.z) * n * k;
    C += int64_t(blockIdx.z) * m * n;
    if (D) D += int64_t(blockIdx.z) * m * n;
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < k; k0 += 16) {
        for (int i = threadIdx.x; i < 1024; i += 256) {
            const int kk = i % 16, r = i / 16;
            sa[kk][r] = r0 + r < m && k0 + kk < k ? A[int64_t(r0 + r) * k + k0 + kk] : 0.f;
            if (TB)
                sb[kk][r] = c0 + r < n && k0 + kk < k ? B[int64_t(c0 + r) * k + k0 + kk] : 0.f;
            else
                sb[i / 64][i % 64] = c0 + i % 64 < n && k0 + i / 64 < k ? B[int64_t(k0 + i / 64) * n + c0 + i % 64] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[kk][ty * 4 + i], sb[kk][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int r = r0 + ty * 4 + i, c = c0 + tx * 4 + j;
            if (r < m && c < n) C[int64_t(r) * n + c] = alpha * acc[i][j] + (D ? beta * D[int64_t(r) * n + c] : 0.f);
        }
}

struct Parts {
    float *inv, *x[2], *p, *q;
    size_t bytes;
};
Parts parts_of(const OrthoShape& s, void* ws) {
    const size_t m = std::min(s.rows, s.cols), n = std::max(s.rows, s.cols), b = s.n_matrices;
    char* at = static_cast<char*>(ws);
    size_t used = 0;
    auto take = [&](size_t count) {
        float* r = reinterpret_cast<float*>(at + used);
        used += align256(count * 4);
        return r;
    };
    Parts p;
    p.inv = take(b);
    p.x[0] = take(b * m * n);
    p.x[1] = take(b * m * n);
    p.p = take(b * m * m);
    p.q = take(b * m * m);
    p.bytes = used;
    return p;
}

template <typename T>
cudaError_t run(const OrthoShape& s, const void* g, void* out, void* ws, cudaStream_t st) {
    const Parts p = parts_of(s, ws);
    const bool turned = s.rows > s.cols;
    const int m = std::min(s.rows, s.cols), n = std::max(s.rows, s.cols), b = s.n_matrices;
    const dim3 flat(unsigned(std::min<int64_t>((int64_t(m) * n + 255) / 256, 1024)), b);
    const T* gp = static_cast<const T*>(g);
    norm_kernel<T><<<b, 512, 0, st>>>(s.rows, s.cols, s.g_matrix, s.g_row, float(s.eps), gp, p.inv);
    take_kernel<T><<<flat, 256, 0, st>>>(m, n, turned, s.g_matrix, s.g_row, gp, p.inv, p.x[0]);
    const dim3 square((m + 63) / 64, (m + 63) / 64, b), wide((n + 63) / 64, (m + 63) / 64, b);
    for (int i = 0; i < s.steps; ++i) {
        const float *x = p.x[i & 1], *none = nullptr;
        product_kernel<true><<<square, 256, 0, st>>>(m, m, n, x, x, 1.f, none, 0.f, p.p);
        product_kernel<true><<<square, 256, 0, st>>>(m, m, m, p.p, p.p, float(s.c), p.p, float(s.b), p.q);
        product_kernel<false><<<wide, 256, 0, st>>>(m, n, m, p.q, x, 1.f, x, float(s.a), p.x[(i + 1) & 1]);
    }
    give_kernel<T><<<flat, 256, 0, st>>>(m, n, turned, s.o_matrix, s.o_row, float(s.scale), p.x[s.steps & 1], static_cast<T*>(out));
    return cudaGetLastError();
}

}  // namespace

size_t ortho_workspace(const OrthoShape& s) { return s.n_matrices == 0 ? 0 : parts_of(s, nullptr).bytes; }

cudaError_t launch_ortho(const OrthoShape& s, const void* g, void* out, void* ws, int sms, cudaStream_t st) {
    (void)sms;
    switch (s.dtype) {
        case UVU_F32: return run<float>(s, g, out, ws, st);
        case UVU_BF16: return run<__nv_bfloat16>(s, g, out, ws, st);
        case UVU_F16: return run<__half>(s, g, out, ws, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace uvu
