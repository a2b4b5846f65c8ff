// Group norm with an activation, channels last, over a packed batch of graphs.
//
// Rows offsets[b] .. offsets[b+1] of x [N][C] are the nodes of graph b; group g holds the cg = C/G
// channels g cg .. (g+1) cg.  With m = n_b cg values per (graph, group):
//     mean = sum x / m,  rstd = (sum (x - mean)^2 / m + eps)^-1/2,  z = (x - mean) rstd gamma + beta,  y = act(z)
// and, for the cotangent dy, with xh = (x - mean) rstd, dz = dy act'(z), t = dz gamma:
//     dgamma = sum_rows dz xh,  dbeta = sum_rows dz,  dx = rstd (t - mean_bg(t) - xh mean_bg(t xh)).
// The two means of t follow from the per-channel sums of the same graph, sum_c gamma_c sum_n dz and
// sum_c gamma_c sum_n dz xh, so one pass of per-channel sums serves dx, dgamma and dbeta.
//
// Statistics and sums are fp32; a variance is summed about its own mean (a second pass over the
// rows that are in shared memory, or Chan's merge of tiles), never as E[x^2] - mean^2.
//
// Tiles: a row tile holds at most R rows of one graph.  Tile number t(b) = offsets[b] / R + b is
// monotone in b and leaves each graph at least ceil(n_b / R) numbers, so a grid of N / R + B tiles
// covers any batch without a list of lengths; the spare numbers are empty.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstdint>

#include "elem.h"
#include "plan.h"

namespace uvu {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kElemChunk = 4;  // vectors a thread of the elementwise kernels has in flight

struct NormArgs {
    int64_t rows;       // N
    int graphs, C, G, per;  // per = C / G
    int R;              // rows of a tile
    float eps;
    const int32_t* offsets;
    const float *gamma, *beta;
    float *mean, *rstd;  // [B][G]
};

__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// act(z) and act'(z)
template <int ACT>
__device__ __forceinline__ float act_of(float z) {
    return ACT == UVU_ACT_SILU ? z * sigmoid(z) : z;
}
template <int ACT>
__device__ __forceinline__ float dact_of(float z) {
    if (ACT != UVU_ACT_SILU) return 1.f;
    const float s = sigmoid(z);
    return s * (1.f + z * (1.f - s));
}

// The graph of tile `t` by the numbering above, or -1 for a spare number; rows [r0, r1).
__device__ __forceinline__ int tile_graph(const int32_t* offsets, int graphs, int R, int64_t t, int64_t& r0, int64_t& r1) {
    int lo = 0, hi = graphs;  // the last b with t(b) <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (int64_t(offsets[mid]) / R + mid <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int64_t a = offsets[lo], e = offsets[lo + 1];
    r0 = a + (t - (a / R + lo)) * R;
    r1 = min(r0 + R, e);
    return r0 < r1 ? lo : -1;
}

// Sums of f over the block's rows, per channel of its slab, in s_chan[0 .. SC): the threads of a
// row take consecutive vectors; kThreads / lanes rows go in parallel and are then added in order.
template <int V, int NS, typename F>
__device__ __forceinline__ void channel_sums(int rows, int SC, float* s_part, float* s_chan, F f) {
    const int vecs = SC / V;
    const int lanes = min(vecs, kThreads), par = kThreads / lanes;
    const int rl = threadIdx.x / lanes, cl = threadIdx.x - rl * lanes;
    for (int cv0 = 0; cv0 < vecs; cv0 += lanes) {
        const int cv = cv0 + cl;
        const int width = min(lanes, vecs - cv0) * V;
        if (rl < par && cv < vecs) {
            float acc[NS][V];
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[s][i] = 0.f;
            for (int r = rl; r < rows; r += par) f(r, cv * V, acc);
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int i = 0; i < V; ++i) s_part[(s * par + rl) * width + cl * V + i] = acc[s][i];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < width * NS; c += kThreads) {
            const int s = c / width, cc = c - s * width;
            float sum = 0.f;
            for (int k = 0; k < par; ++k) sum += s_part[(s * par + k) * width + cc];
            s_chan[s * SC + cv0 * V + cc] = sum;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------- tiles

// Forward, pass 1: mean and centred sum of squares of each (tile, group), ws[t][G][2].
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_tile_stats(NormArgs a, const T* __restrict__ x, float* __restrict__ ws) {
    extern __shared__ __align__(16) float smem[];
    float* s_part = smem;                 // [kThreads * V]
    float* s_chan = s_part + max(kThreads * V, a.C);
    float* s_mean = s_chan + a.C;
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, blockIdx.x, r0, r1);
    if (b < 0) return;
    const int rows = int(r1 - r0);
    const T* xt = x + r0 * a.C;
    channel_sums<V, 1>(rows, a.C, s_part, s_chan, [&](int r, int c, float (&acc)[1][V]) {
        const Vec<T, V> v = load_vec<T, V>(xt + int64_t(r) * a.C + c);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[0][i] += widen(v.v[i]);
    });
    const float inv = 1.f / (float(rows) * float(a.per));
    for (int g = threadIdx.x; g < a.G; g += kThreads) {
        float s = 0.f;
        for (int c = 0; c < a.per; ++c) s += s_chan[g * a.per + c];
        s_mean[g] = s * inv;
    }
    __syncthreads();
    channel_sums<V, 1>(rows, a.C, s_part, s_chan, [&](int r, int c, float (&acc)[1][V]) {
        const Vec<T, V> v = load_vec<T, V>(xt + int64_t(r) * a.C + c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float d = widen(v.v[i]) - s_mean[(c + i) / a.per];
            acc[0][i] = fmaf(d, d, acc[0][i]);
        }
    });
    for (int g = threadIdx.x; g < a.G; g += kThreads) {
        float s = 0.f;
        for (int c = 0; c < a.per; ++c) s += s_chan[g * a.per + c];
        float* o = ws + (int64_t(blockIdx.x) * a.G + g) * 2;
        o[0] = s_mean[g];
        o[1] = s;
    }
}

// Forward, pass 2: Chan's merge of a graph's tiles, one warp per (graph, group): each lane merges
// every 32nd tile in order, then the lanes pairwise.
__global__ void __launch_bounds__(128) norm_merge(NormArgs a, const float* __restrict__ ws) {
    const int64_t i = (int64_t(blockIdx.x) * 128 + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (i >= int64_t(a.graphs) * a.G) return;
    const int b = int(i / a.G), g = int(i % a.G);
    const int64_t r0 = a.offsets[b], n = a.offsets[b + 1] - r0;
    const int64_t t0 = r0 / a.R + b, tiles = (n + a.R - 1) / a.R;
    float cnt = 0.f, mean = 0.f, m2 = 0.f;
    auto merge = [&](float c2, float mean2, float m22) {
        const float tot = cnt + c2;
        if (c2 > 0.f) {
            const float d = mean2 - mean, w = c2 / tot;
            mean = fmaf(d, w, mean);
            m2 += m22 + d * d * cnt * w;
            cnt = tot;
        }
    };
    for (int64_t t = lane; t < tiles; t += 32) {
        const float* o = ws + ((t0 + t) * a.G + g) * 2;
        merge(float(min(int64_t(a.R), n - t * a.R)) * float(a.per), o[0], o[1]);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) {
        const float c2 = __shfl_down_sync(0xffffffffu, cnt, k), u = __shfl_down_sync(0xffffffffu, mean, k),
                    w = __shfl_down_sync(0xffffffffu, m2, k);
        merge(c2, u, w);
    }
    if (lane == 0) {
        a.mean[i] = mean;
        a.rstd[i] = rsqrtf((cnt > 0.f ? m2 / cnt : 0.f) + a.eps);
    }
}

// Forward, pass 3: y.  One tile per block.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_apply(NormArgs a, const T* __restrict__ x, T* __restrict__ y) {
    extern __shared__ __align__(16) float smem[];
    float *s_a = smem, *s_mean = smem + a.C;  // z = (x - mean) s_a + beta: a folded x s_a + b would cancel where rstd is large
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, blockIdx.x, r0, r1);
    if (b < 0) return;
    for (int c = threadIdx.x; c < a.C; c += kThreads) {
        const int64_t i = int64_t(b) * a.G + c / a.per;
        s_a[c] = a.rstd[i] * a.gamma[c];
        s_mean[c] = a.mean[i];
    }
    __syncthreads();
    const int vecs = a.C / V;
    const int64_t total = (r1 - r0) * vecs;
    const T* xt = x + r0 * a.C;
    T* yt = y + r0 * a.C;
    for (int64_t k = threadIdx.x; k < total; k += kThreads) {
        const int c = int(k % vecs) * V;
        const Vec<T, V> v = load_vec<T, V>(xt + k * V);
        Vec<T, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) o.v[i] = narrow<T>(act_of<ACT>(fmaf(widen(v.v[i]) - s_mean[c + i], s_a[c + i], a.beta[c + i])));
        store_vec<T, V>(yt + k * V, o);
    }
}

// Backward, pass 1: per-channel sums of dz and dz xh of each tile, ws[t][2][C].
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_bwd_tile_sums(NormArgs a, const T* __restrict__ x, const T* __restrict__ dy,
                                                               float* __restrict__ ws) {
    extern __shared__ __align__(16) float smem[];
    float* s_part = smem;  // [2 * kThreads * V]
    float* s_chan = s_part + 2 * max(kThreads * V, a.C);
    float *s_mean = s_chan + 2 * a.C, *s_rstd = s_mean + a.G;
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, blockIdx.x, r0, r1);
    if (b < 0) return;
    for (int g = threadIdx.x; g < a.G; g += kThreads) {
        s_mean[g] = a.mean[int64_t(b) * a.G + g];
        s_rstd[g] = a.rstd[int64_t(b) * a.G + g];
    }
    __syncthreads();
    const T *xt = x + r0 * a.C, *gt = dy + r0 * a.C;
    channel_sums<V, 2>(int(r1 - r0), a.C, s_part, s_chan, [&](int r, int c, float (&acc)[2][V]) {
        const Vec<T, V> v = load_vec<T, V>(xt + int64_t(r) * a.C + c), d = load_vec<T, V>(gt + int64_t(r) * a.C + c);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int g = (c + i) / a.per;
            const float xh = (widen(v.v[i]) - s_mean[g]) * s_rstd[g];
            const float dz = widen(d.v[i]) * dact_of<ACT>(fmaf(xh, a.gamma[c + i], a.beta[c + i]));
            acc[0][i] += dz;
            acc[1][i] = fmaf(dz, xh, acc[1][i]);
        }
    });
    float* o = ws + int64_t(blockIdx.x) * 2 * a.C;
    for (int c = threadIdx.x; c < 2 * a.C; c += kThreads) o[c] = s_chan[c];
}

// Backward, pass 2: a graph's channel sums over its tiles (in order) to sums[b][2][C].
__global__ void __launch_bounds__(kThreads) norm_bwd_merge(NormArgs a, const float* __restrict__ ws, float* __restrict__ sums) {
    const int b = blockIdx.x;
    const int c = blockIdx.y * kThreads + threadIdx.x;
    if (c >= 2 * a.C) return;
    const int64_t r0 = a.offsets[b], n = a.offsets[b + 1] - r0;
    const int64_t t0 = r0 / a.R + b, tiles = (n + a.R - 1) / a.R;
    float s = 0.f;
    for (int64_t t = 0; t < tiles; ++t) s += ws[(t0 + t) * 2 * a.C + c];
    sums[int64_t(b) * 2 * a.C + c] = s;
}

// Backward, pass 3: dx of a tile.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_bwd_apply(NormArgs a, const T* __restrict__ x, const T* __restrict__ dy,
                                                           const float* __restrict__ sums, T* __restrict__ dx) {
    extern __shared__ __align__(16) float smem[];
    float *s_m1 = smem, *s_m2 = s_m1 + a.G, *s_mean = s_m2 + a.G, *s_rstd = s_mean + a.G;
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, blockIdx.x, r0, r1);
    if (b < 0) return;
    const float inv = 1.f / (float(a.offsets[b + 1] - a.offsets[b]) * float(a.per));
    for (int g = threadIdx.x; g < a.G; g += kThreads) {
        float p = 0.f, q = 0.f;
        const float* o = sums + int64_t(b) * 2 * a.C + g * a.per;
        for (int c = 0; c < a.per; ++c) {
            p = fmaf(a.gamma[g * a.per + c], o[c], p);
            q = fmaf(a.gamma[g * a.per + c], o[a.C + c], q);
        }
        s_m1[g] = p * inv;
        s_m2[g] = q * inv;
        s_mean[g] = a.mean[int64_t(b) * a.G + g];
        s_rstd[g] = a.rstd[int64_t(b) * a.G + g];
    }
    __syncthreads();
    const int vecs = a.C / V;
    const int64_t total = (r1 - r0) * vecs;
    const T *xt = x + r0 * a.C, *gt = dy + r0 * a.C;
    T* ot = dx + r0 * a.C;
    for (int64_t k = threadIdx.x; k < total; k += kThreads) {
        const int c = int(k % vecs) * V;
        const Vec<T, V> v = load_vec<T, V>(xt + k * V), d = load_vec<T, V>(gt + k * V);
        Vec<T, V> o;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int g = (c + i) / a.per;
            const float gam = a.gamma[c + i];
            const float xh = (widen(v.v[i]) - s_mean[g]) * s_rstd[g];
            const float t = widen(d.v[i]) * dact_of<ACT>(fmaf(xh, gam, a.beta[c + i])) * gam;
            o.v[i] = narrow<T>(s_rstd[g] * (t - s_m1[g] - xh * s_m2[g]));
        }
        store_vec<T, V>(ot + k * V, o);
    }
}

// Backward, pass 4: dgamma and dbeta, the sums of the graphs' channel sums.  One warp per channel
// of the 2 C sums, lanes over the graphs, then pairwise.
__global__ void __launch_bounds__(256) norm_bwd_params(int graphs, int C, const float* __restrict__ sums,
                                                       float* __restrict__ dgamma, float* __restrict__ dbeta) {
    __shared__ float s[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // coalesced over channels; the warps share the graphs
    float acc = 0.f;
    if (c < 2 * C)
        for (int b = w; b < graphs; b += 8) acc += sums[int64_t(b) * 2 * C + c];
    s[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < 2 * C) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += s[k][lane];
        if (c < C)
            dbeta[c] = t;
        else
            dgamma[c - C] = t;
    }
}

// Rows of a tile: about 32 KB of x, 16 rows at least.
int tile_rows(int C, size_t elem) { return int(std::min<size_t>(4096, std::max<size_t>(16, 32768 / (size_t(C) * elem)))); }

struct Plan2 {
    int R;
    int64_t tiles;
};
Plan2 plan_tiles(int64_t N, int B, int C, size_t elem) {
    Plan2 p;
    p.R = tile_rows(C, elem);
    p.tiles = N / p.R + B;
    return p;
}

size_t dtype_bytes(uvu_dtype t) { return t == UVU_F32 ? 4 : 2; }
size_t align256(size_t b) { return (b + 255) / 256 * 256; }

template <typename T, int V, int ACT>
cudaError_t fwd(NormArgs a, const T* x, T* y, float* ws, cudaStream_t st) {
    const Plan2 p = plan_tiles(a.rows, a.graphs, a.C, sizeof(T));
    a.R = p.R;
    const size_t sm = (size_t(std::max(kThreads * V, a.C)) + a.C + a.G) * 4;
    cudaError_t e = cudaFuncSetAttribute(norm_tile_stats<T, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sm));
    if (e != cudaSuccess) return e;
    norm_tile_stats<T, V><<<unsigned(p.tiles), kThreads, sm, st>>>(a, x, ws);
    norm_merge<<<unsigned((int64_t(a.graphs) * a.G + 3) / 4), 128, 0, st>>>(a, ws);
    e = cudaFuncSetAttribute(norm_apply<T, V, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, a.C * 8);
    if (e != cudaSuccess) return e;
    norm_apply<T, V, ACT><<<unsigned(p.tiles), kThreads, size_t(a.C) * 8, st>>>(a, x, y);
    return cudaGetLastError();
}

template <typename T, int V, int ACT>
cudaError_t bwd(NormArgs a, const T* x, const T* dy, T* dx, float* dgamma, float* dbeta, float* ws, cudaStream_t st) {
    const Plan2 p = plan_tiles(a.rows, a.graphs, a.C, sizeof(T));
    a.R = p.R;
    float* sums = ws + align256(size_t(p.tiles) * 2 * a.C * 4) / 4;
    if (a.rows > 0) {
        const size_t sm = (size_t(std::max(kThreads * V, a.C)) * 2 + 2 * size_t(a.C) + 2 * size_t(a.G)) * 4;
        cudaError_t e = cudaFuncSetAttribute(norm_bwd_tile_sums<T, V, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sm));
        if (e != cudaSuccess) return e;
        norm_bwd_tile_sums<T, V, ACT><<<unsigned(p.tiles), kThreads, sm, st>>>(a, x, dy, ws);
    }
    norm_bwd_merge<<<dim3(unsigned(a.graphs), unsigned((2 * a.C + kThreads - 1) / kThreads)), kThreads, 0, st>>>(a, ws, sums);
    if (a.rows > 0)
        norm_bwd_apply<T, V, ACT><<<unsigned(p.tiles), kThreads, size_t(a.G) * 16, st>>>(a, x, dy, sums, dx);
    norm_bwd_params<<<unsigned((2 * a.C + 31) / 32), 256, 0, st>>>(a.graphs, a.C, sums, dgamma, dbeta);
    return cudaGetLastError();
}

// 16-byte vectors when every row begins on a 16-byte boundary, else single elements.
template <typename T, typename F>
cudaError_t by_vector(int C, uintptr_t any, F f) {
    if (C % int(16 / sizeof(T)) == 0 && (any & 15u) == 0) return f(std::integral_constant<int, int(16 / sizeof(T))>{});
    return f(std::integral_constant<int, 1>{});
}

template <typename T>
cudaError_t fwd_of(const NormArgs& a, uvu_act act, const void* x, void* y, void* ws, cudaStream_t st) {
    return by_vector<T>(a.C, reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y), [&](auto v) {
        constexpr int V = decltype(v)::value;
        const T* xp = static_cast<const T*>(x);
        T* yp = static_cast<T*>(y);
        float* w = static_cast<float*>(ws);
        return act == UVU_ACT_SILU ? fwd<T, V, UVU_ACT_SILU>(a, xp, yp, w, st) : fwd<T, V, UVU_ACT_NONE>(a, xp, yp, w, st);
    });
}
template <typename T>
cudaError_t bwd_of(const NormArgs& a, uvu_act act, const void* x, const void* dy, void* dx, float* dg, float* db, void* ws,
                   cudaStream_t st) {
    const uintptr_t any = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(dx);
    return by_vector<T>(a.C, any, [&](auto v) {
        constexpr int V = decltype(v)::value;
        const T *xp = static_cast<const T*>(x), *gp = static_cast<const T*>(dy);
        T* op = static_cast<T*>(dx);
        float* w = static_cast<float*>(ws);
        return act == UVU_ACT_SILU ? bwd<T, V, UVU_ACT_SILU>(a, xp, gp, op, dg, db, w, st)
                                   : bwd<T, V, UVU_ACT_NONE>(a, xp, gp, op, dg, db, w, st);
    });
}

NormArgs norm_args(const NormShape& s, const int32_t* offsets, const float* gamma, const float* beta, float* mean, float* rstd) {
    NormArgs a;
    a.rows = s.rows;
    a.graphs = s.graphs;
    a.C = s.channels;
    a.G = s.groups;
    a.per = s.channels / s.groups;
    a.R = 0;
    a.eps = float(s.eps);
    a.offsets = offsets;
    a.gamma = gamma;
    a.beta = beta;
    a.mean = mean;
    a.rstd = rstd;
    return a;
}

}  // namespace

size_t norm_workspace(const NormShape& s, bool bwd) {
    const Plan2 p = plan_tiles(s.rows, s.graphs, s.channels, dtype_bytes(s.dtype));
    if (!bwd) return size_t(p.tiles) * s.groups * 8;
    return align256(size_t(p.tiles) * 2 * s.channels * 4) + size_t(s.graphs) * 2 * s.channels * 4;
}

cudaError_t launch_norm_fwd(const NormShape& s, const int32_t* offsets, const void* x, const float* gamma, const float* beta,
                            void* y, float* mean, float* rstd, void* ws, cudaStream_t st) {
    const NormArgs a = norm_args(s, offsets, gamma, beta, mean, rstd);
    switch (s.dtype) {
        case UVU_F32: return fwd_of<float>(a, s.act, x, y, ws, st);
        case UVU_BF16: return fwd_of<__nv_bfloat16>(a, s.act, x, y, ws, st);
        case UVU_F16: return fwd_of<__half>(a, s.act, x, y, ws, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_norm_bwd(const NormShape& s, const int32_t* offsets, const void* x, const void* dy, const float* gamma,
                            const float* beta, const float* mean, const float* rstd, void* dx, float* dgamma, float* dbeta,
                            void* ws, cudaStream_t st) {
    const NormArgs a = norm_args(s, offsets, gamma, beta, const_cast<float*>(mean), const_cast<float*>(rstd));
    switch (s.dtype) {
        case UVU_F32: return bwd_of<float>(a, s.act, x, dy, dx, dgamma, dbeta, ws, st);
        case UVU_BF16: return bwd_of<__nv_bfloat16>(a, s.act, x, dy, dx, dgamma, dbeta, ws, st);
        case UVU_F16: return bwd_of<__half>(a, s.act, x, dy, dx, dgamma, dbeta, ws, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace uvu
