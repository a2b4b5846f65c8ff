// Group norm with an activation, channels last, over a packed batch of graphs.
//
// Rows offsets[b] .. offsets[b+1] of x [N][C] are the nodes of graph b; group g holds the per = C/G
// channels g per .. (g+1) per.  With m = n_b per values per (graph, group):
//     mean = sum x / m,  rstd = (sum (x - mean)^2 / m + eps)^-1/2,  z = (x - mean) rstd gamma + beta,  y = act(z)
// and, for the cotangent dy, with xh = (x - mean) rstd, dz = dy act'(z), t = dz gamma:
//     dgamma = sum_rows dz xh,  dbeta = sum_rows dz,  dx = rstd (t - mean_bg(t) - xh mean_bg(t xh)).
// The two means of t follow from the per-channel sums of the same graph, sum_c gamma_c sum_n dz and
// sum_c gamma_c sum_n dz xh, so one pass of per-channel sums serves dx, dgamma and dbeta.
//
// Statistics and sums are fp32; a variance is summed about its own mean (a second pass over rows
// that are in shared memory, or Chan's merge of tiles), never as E[x^2] - mean^2.
//
// Bound by memory: x (and dy) in, y (or dx) out.  Two forms:
//   - on chip: a cluster of 1 .. 8 blocks holds one graph's rows of a slab of channels (whole groups,
//     at least 128 bytes of a row) in shared memory, adds its sums through distributed shared memory
//     and writes the result: each value crosses HBM once each way.  Taken when the longest graph
//     fits (max_rows; rows beyond it are read again from memory, so a wrong max_rows costs time only).
//   - tiled: for longer graphs, row tiles to per-tile statistics, a merge per graph, and a second
//     pass that walks the tiles backwards, so that what L2 still holds is read there.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstdint>
#include <numeric>

#include "elem.h"
#include "plan.h"

namespace uvu {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;

struct NormArgs {
    int64_t rows;        // N
    int graphs, C, G, per;  // per = C / G
    int R;               // rows of a tile, or of a block's share that shared memory holds
    int slab, slabs;     // channels of a block (on-chip form), slabs of C
    float eps;
    const int32_t* offsets;
    const float *gamma, *beta;
    float *mean, *rstd;  // [B][G]
};

// Pairs of fp32 values: one packed instruction does both (add, mul, fma .f32x2), which halves the
// arithmetic that a value costs beside the two special-function instructions of its sigmoid.
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

// The pairs of a vector; a single element is paired with zero.
template <int V>
constexpr int kPairs = V > 1 ? V / 2 : 1;
template <typename T, int V>
__device__ __forceinline__ F2 pair_of(const Vec<T, V>& v, int i) {
    return F2(widen(v.v[2 * i]), V > 1 ? widen(v.v[V > 1 ? 2 * i + 1 : 0]) : 0.f);
}
template <typename T, int V>
__device__ __forceinline__ void put_pair(Vec<T, V>& v, int i, F2 x) {
    const float2 b = x.both();
    v.v[2 * i] = narrow<T>(b.x);
    if (V > 1) v.v[V > 1 ? 2 * i + 1 : 0] = narrow<T>(b.y);
}

__device__ __forceinline__ float exp2f_fast(float x) {  // 2^x, 2 ulp
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + exp(-z)).  __fdividef's result is 0 for a denominator above 2^126: the sigmoid is below 2^-126 there.
__device__ __forceinline__ F2 sigmoid(F2 z) {
    const float2 e = (z * F2(-1.4426950408889634f, -1.4426950408889634f)).both();
    const float2 d = (F2(exp2f_fast(e.x), exp2f_fast(e.y)) + F2(1.f, 1.f)).both();
    return F2(__fdividef(1.f, d.x), __fdividef(1.f, d.y));
}

// act(z), and dy act'(z)
template <int ACT>
__device__ __forceinline__ F2 act_of(F2 z) {
    return ACT == UVU_ACT_SILU ? z * sigmoid(z) : z;
}
template <int ACT>
__device__ __forceinline__ F2 dact_of(F2 dy, F2 z) {
    if (ACT != UVU_ACT_SILU) return dy;
    const F2 s = sigmoid(z), one(1.f, 1.f), minus(-1.f, -1.f);
    return dy * (s * fma2(z, fma2(s, minus, one), one));
}

// Rows [r0, r1) of tile `t` and its graph, or -1 for a spare number: tile t(b) = offsets[b] / R + b is
// monotone in b and leaves each graph at least ceil(n_b / R) numbers, so a grid of N / R + B tiles
// covers any batch without a list of lengths.
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

// The block's threads over `vecs` vectors of a row: consecutive threads take consecutive vectors, and
// kThreads / lanes rows go in parallel.  f(cv, rl, par): vector cv of the rows rl, rl + par, ...;
// rows wider than the block take several rounds.  after(cv0, width): between rounds, by all threads.
template <typename F, typename A>
__device__ __forceinline__ void over_columns(int vecs, F f, A after) {
    const int lanes = min(vecs, kThreads), par = kThreads / lanes;
    const int rl = threadIdx.x / lanes, cl = threadIdx.x - rl * lanes;
    for (int cv0 = 0; cv0 < vecs; cv0 += lanes) {
        if (rl < par && cv0 + cl < vecs) f(cv0 + cl, rl, par);
        after(cv0, min(lanes, vecs - cv0), par);
    }
}

// The group of each channel of a vector, from one division.
template <int V, typename F>
__device__ __forceinline__ void each_channel(int c0, int per, F f) {
    int g = c0 / per, left = per - (c0 - g * per);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (left == 0) ++g, left = per;
        f(i, g);
        --left;
    }
}
// A value per channel of a vector, as pairs.
template <int V>
struct Channels {
    F2 v[kPairs<V>];
    template <typename F>
    __device__ __forceinline__ void set(int c0, int per, F f) {
        float x[2 * kPairs<V>];
        x[2 * kPairs<V> - 1] = 0.f;
        each_channel<V>(c0, per, [&](int i, int g) { x[i] = f(i, g); });
#pragma unroll
        for (int i = 0; i < kPairs<V>; ++i) v[i] = F2(x[2 * i], x[2 * i + 1]);
    }
};

// NS sums per channel over `rows` rows, to s_chan[s * SC + c].  f(cv) gives the function of (row, acc)
// that adds a row's terms for vector cv.
template <int V, int NS, typename F>
__device__ __forceinline__ void channel_sums(int rows, int SC, float* s_part, float* s_chan, F f) {
    const int lanes = min(SC / V, kThreads), width = lanes * V;
    over_columns(
        SC / V,
        [&](int cv, int rl, int par) {
            F2 acc[NS][kPairs<V>];
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int i = 0; i < kPairs<V>; ++i) acc[s][i] = F2(0.f, 0.f);
            auto add = f(cv);
#pragma unroll 1
            for (int r = rl; r < rows; r += par) add(r, acc);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                float* o = s_part + (s * par + rl) * width + (cv % lanes) * V;
                if constexpr (V == 1) {
                    *o = acc[s][0].both().x;
                } else {
#pragma unroll
                    for (int i = 0; i < V / 4; ++i) {
                        const float2 p = acc[s][2 * i].both(), q = acc[s][2 * i + 1].both();
                        reinterpret_cast<float4*>(o)[i] = make_float4(p.x, p.y, q.x, q.y);
                    }
                }
            }
        },
        [&](int cv0, int n, int par) {
            __syncthreads();
            for (int c = threadIdx.x; c < n * V * NS; c += kThreads) {
                const int s = c / (n * V), cc = c - s * n * V;
                const float* p = s_part + s * par * width + cc;
                float sum[2] = {0.f, 0.f};
                int k = 0;
#pragma unroll 4
                for (; k + 1 < par; k += 2) sum[0] += p[k * width], sum[1] += p[(k + 1) * width];
                if (k < par) sum[0] += p[k * width];
                s_chan[s * SC + cv0 * V + cc] = sum[0] + sum[1];
            }
            __syncthreads();
        });
}

// Sums of `per` consecutive channel values per group; 4 lanes of a warp share a group.
template <typename F>
__device__ __forceinline__ void group_sums(int groups, int per, const float* s_chan, F out) {
    for (int g0 = 0; g0 < groups; g0 += kThreads / 4) {
        const int g = g0 + threadIdx.x / 4, l = threadIdx.x & 3;
        float s = 0.f;
        if (g < groups)
            for (int c = l; c < per; c += 4) s += s_chan[g * per + c];
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (g < groups && l == 0) out(g, s);
    }
}

// One vector from global to shared memory, without passing registers where it is 16 bytes.
template <typename T, int V>
__device__ __forceinline__ void stage_vec(T* dst, const T* src) {
    if constexpr (V * sizeof(T) == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(uint32_t(__cvta_generic_to_shared(dst))), "l"(src) : "memory");
    } else {
        *dst = *src;
    }
}
template <typename T, int V>
__device__ __forceinline__ void stage_rows(T* s, const T* x, int rows, int SC, int64_t C) {
    over_columns(
        SC / V,
        [&](int cv, int rl, int par) {
#pragma unroll 4
            for (int r = rl; r < rows; r += par) stage_vec<T, V>(s + r * SC + cv * V, x + r * C + cv * V);
        },
        [](int, int, int) {});
}
__device__ __forceinline__ void stage_wait() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
}

// ----------------------------------------------------------------------------------- on chip

struct Share {  // a block's part of a graph
    int b, c0, SC, rank, rows;
    int K;  // blocks that have rows (one, if none has); the others leave at once
    int64_t n, r0;
};
__device__ __forceinline__ Share share_of(const NormArgs& a) {
    Share s;
    s.K = int(cg::this_cluster().num_blocks());
    s.rank = int(cg::this_cluster().block_rank());
    const int id = int(blockIdx.x) / s.K;
    s.b = id / a.slabs;
    s.c0 = (id - s.b * a.slabs) * a.slab;
    s.SC = min(a.slab, a.C - s.c0);
    const int64_t first = a.offsets[s.b];
    s.n = a.offsets[s.b + 1] - first;
    // whole shares in rank order, so that short graphs need fewer blocks; a graph longer than max_rows
    // promised is shared out evenly
    const int64_t each = max(int64_t(a.R), (s.n + s.K - 1) / s.K), lo = min(s.n, s.rank * each);
    s.r0 = first + lo;
    s.rows = int(min(s.n, lo + each) - lo);
    s.K = int(max(int64_t(1), (s.n + each - 1) / each));
    return s;
}

// s_group[i] (i < count) summed over the cluster's blocks in rank order, to s_sum.
__device__ __forceinline__ void cluster_sums(int count, int K, float* s_group, float* s_sum) {
    if (K == 1) {
        __syncthreads();
        for (int i = threadIdx.x; i < count; i += kThreads) s_sum[i] = s_group[i];
    } else {
        cg::cluster_group c = cg::this_cluster();
        __syncwarp();
        c.sync();
        for (int i = threadIdx.x; i < count; i += kThreads) {
            float s = 0.f;
            for (int k = 0; k < K; ++k) s += c.map_shared_rank(s_group, k)[i];
            s_sum[i] = s;
        }
    }
    __syncthreads();
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_fwd_chip(NormArgs a, const T* __restrict__ x, T* __restrict__ y) {
    extern __shared__ __align__(16) unsigned char smem[];
    const Share s = share_of(a);
    if (s.rank >= s.K) return;
    const int groups = s.SC / a.per, g0 = s.c0 / a.per;
    T* s_x = reinterpret_cast<T*>(smem);
    float* s_part = reinterpret_cast<float*>(smem + (size_t(a.R) * a.slab * sizeof(T) + 15) / 16 * 16);
    float *s_chan = s_part + max(kThreads * V, a.slab), *s_g1 = s_chan + a.slab, *s_g2 = s_g1 + a.slab / a.per,
          *s_mean = s_g2 + a.slab / a.per, *s_rstd = s_mean + a.slab / a.per;
    const T* xs = x + s.r0 * a.C + s.c0;
    const int held = min(s.rows, a.R);
    stage_rows<T, V>(s_x, xs, held, s.SC, a.C);
    stage_wait();
    auto row = [&](int r, int cv) {
        return load_vec<T, V>(r < held ? s_x + r * s.SC + cv * V : xs + int64_t(r) * a.C + cv * V);
    };
    channel_sums<V, 1>(s.rows, s.SC, s_part, s_chan, [&](int cv) {
        return [&, cv](int r, F2 (&acc)[1][kPairs<V>]) {
            const Vec<T, V> v = row(r, cv);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) acc[0][i] = acc[0][i] + pair_of(v, i);
        };
    });
    group_sums(groups, a.per, s_chan, [&](int g, float v) { s_g1[g] = v; });
    cluster_sums(groups, s.K, s_g1, s_mean);
    const float inv = s.n > 0 ? 1.f / (float(s.n) * float(a.per)) : 0.f;
    channel_sums<V, 1>(s.rows, s.SC, s_part, s_chan, [&](int cv) {
        Channels<V> minus;
        minus.set(cv * V, a.per, [&](int, int g) { return -s_mean[g] * inv; });
        return [&, cv, minus](int r, F2 (&acc)[1][kPairs<V>]) {
            const Vec<T, V> v = row(r, cv);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) {
                const F2 d = pair_of(v, i) + minus.v[i];
                acc[0][i] = fma2(d, d, acc[0][i]);
            }
        };
    });
    group_sums(groups, a.per, s_chan, [&](int g, float v) { s_g2[g] = v; });
    cluster_sums(groups, s.K, s_g2, s_rstd);
    if (s.K > 1) cg::this_cluster().barrier_arrive();  // the other blocks' sums have been read
    for (int g = threadIdx.x; g < groups; g += kThreads) {
        s_rstd[g] = rsqrtf(s_rstd[g] * inv + a.eps);
        if (s.rank == 0) {
            a.mean[int64_t(s.b) * a.G + g0 + g] = s_mean[g] * inv;
            a.rstd[int64_t(s.b) * a.G + g0 + g] = s_rstd[g];
        }
    }
    __syncthreads();
    T* ys = y + s.r0 * a.C + s.c0;
    over_columns(
        s.SC / V,
        [&](int cv, int rl, int par) {
            Channels<V> minus, k, beta;
            minus.set(cv * V, a.per, [&](int, int g) { return -s_mean[g] * inv; });
            k.set(cv * V, a.per, [&](int i, int g) { return s_rstd[g] * a.gamma[s.c0 + cv * V + i]; });
            beta.set(cv * V, a.per, [&](int i, int) { return a.beta[s.c0 + cv * V + i]; });
#pragma unroll 1
            for (int r = rl; r < s.rows; r += par) {
                const Vec<T, V> v = row(r, cv);
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < kPairs<V>; ++i)
                    put_pair(o, i, act_of<ACT>(fma2(pair_of(v, i) + minus.v[i], k.v[i], beta.v[i])));
                store_vec<T, V>(ys + int64_t(r) * a.C + cv * V, o);
            }
        },
        [](int, int, int) {});
    __syncwarp();
    if (s.K > 1) cg::this_cluster().barrier_wait();
}

// A thread's channels of the backward: xh and dz of a pair of values.
template <int V, int ACT>
struct BwdChannel {
    Channels<V> minus, rstd, gamma, beta;
    __device__ __forceinline__ BwdChannel(const NormArgs& a, int b, int c) {
        const int64_t g0 = int64_t(b) * a.G;
        minus.set(c, a.per, [&](int, int g) { return -a.mean[g0 + g]; });
        rstd.set(c, a.per, [&](int, int g) { return a.rstd[g0 + g]; });
        gamma.set(c, a.per, [&](int i, int) { return a.gamma[c + i]; });
        beta.set(c, a.per, [&](int i, int) { return a.beta[c + i]; });
    }
    __device__ __forceinline__ F2 xh(F2 x, int i) const { return (x + minus.v[i]) * rstd.v[i]; }
    __device__ __forceinline__ F2 dz(F2 dy, F2 xh, int i) const { return dact_of<ACT>(dy, fma2(xh, gamma.v[i], beta.v[i])); }
    __device__ __forceinline__ void add(F2 x, F2 dy, int i, F2& s0, F2& s1) const {
        const F2 h = xh(x, i), d = dz(dy, h, i);
        s0 = s0 + d;
        s1 = fma2(d, h, s1);
    }
    // rstd (dz gamma - m1 - xh m2), with -m1 and -m2
    __device__ __forceinline__ F2 dx(F2 x, F2 dy, int i, F2 m1, F2 m2) const {
        const F2 h = xh(x, i);
        return rstd.v[i] * fma2(h, m2, fma2(dz(dy, h, i), gamma.v[i], m1));
    }
};

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads, 3) norm_bwd_chip(NormArgs a, const T* __restrict__ x, const T* __restrict__ dy,
                                                          T* __restrict__ dx, float* __restrict__ sums) {
    extern __shared__ __align__(16) unsigned char smem[];
    const Share s = share_of(a);
    if (s.rank >= s.K) return;
    const int groups = s.SC / a.per;
    const size_t tile = (size_t(a.R) * a.slab * sizeof(T) + 15) / 16 * 16;
    T *s_x = reinterpret_cast<T*>(smem), *s_d = reinterpret_cast<T*>(smem + tile);
    float* s_part = reinterpret_cast<float*>(smem + 2 * tile);
    float *s_chan = s_part + 2 * max(kThreads * V, a.slab), *s_sum = s_chan + 2 * a.slab, *s_m1 = s_sum + 2 * a.slab,
          *s_m2 = s_m1 + a.slab / a.per;
    const T *xs = x + s.r0 * a.C + s.c0, *ds = dy + s.r0 * a.C + s.c0;
    const int held = min(s.rows, a.R);
    stage_rows<T, V>(s_x, xs, held, s.SC, a.C);
    stage_rows<T, V>(s_d, ds, held, s.SC, a.C);
    stage_wait();
    auto row = [&](const T* sm, const T* gm, int r, int cv) {
        return load_vec<T, V>(r < held ? sm + r * s.SC + cv * V : gm + int64_t(r) * a.C + cv * V);
    };
    channel_sums<V, 2>(s.rows, s.SC, s_part, s_chan, [&](int cv) {
        const BwdChannel<V, ACT> ch(a, s.b, s.c0 + cv * V);
        return [&, cv, ch](int r, F2 (&acc)[2][kPairs<V>]) {
            const Vec<T, V> v = row(s_x, xs, r, cv), d = row(s_d, ds, r, cv);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) ch.add(pair_of(v, i), pair_of(d, i), i, acc[0][i], acc[1][i]);
        };
    });
    cluster_sums(2 * s.SC, s.K, s_chan, s_sum);
    if (s.K > 1) cg::this_cluster().barrier_arrive();  // the other blocks' sums have been read
    if (s.rank == 0)
        for (int c = threadIdx.x; c < 2 * s.SC; c += kThreads)
            sums[int64_t(s.b) * 2 * a.C + (c < s.SC ? s.c0 + c : a.C + s.c0 + c - s.SC)] = s_sum[c];
    for (int c = threadIdx.x; c < 2 * s.SC; c += kThreads) s_part[c] = s_sum[c] * a.gamma[s.c0 + (c < s.SC ? c : c - s.SC)];
    __syncthreads();
    const float inv = s.n > 0 ? 1.f / (float(s.n) * float(a.per)) : 0.f;
    group_sums(groups, a.per, s_part, [&](int g, float v) { s_m1[g] = v * inv; });
    group_sums(groups, a.per, s_part + s.SC, [&](int g, float v) { s_m2[g] = v * inv; });
    __syncthreads();
    T* os = dx + s.r0 * a.C + s.c0;
    over_columns(
        s.SC / V,
        [&](int cv, int rl, int par) {
            const BwdChannel<V, ACT> ch(a, s.b, s.c0 + cv * V);
            Channels<V> m1, m2;
            m1.set(cv * V, a.per, [&](int, int g) { return -s_m1[g]; });
            m2.set(cv * V, a.per, [&](int, int g) { return -s_m2[g]; });
#pragma unroll 1
            for (int r = rl; r < s.rows; r += par) {
                const Vec<T, V> v = row(s_x, xs, r, cv), d = row(s_d, ds, r, cv);
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < kPairs<V>; ++i) put_pair(o, i, ch.dx(pair_of(v, i), pair_of(d, i), i, m1.v[i], m2.v[i]));
                store_vec<T, V>(os + int64_t(r) * a.C + cv * V, o);
            }
        },
        [](int, int, int) {});
    __syncwarp();
    if (s.K > 1) cg::this_cluster().barrier_wait();
}

// ------------------------------------------------------------------------------------- tiles

// Forward, pass 1: mean and centred sum of squares of each (tile, group), ws[t][G][2].
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_tile_stats(NormArgs a, const T* __restrict__ x, float* __restrict__ ws) {
    extern __shared__ __align__(16) unsigned char smem[];
    T* s_x = reinterpret_cast<T*>(smem);
    float* s_part = reinterpret_cast<float*>(smem + (size_t(a.R) * a.C * sizeof(T) + 15) / 16 * 16);
    float *s_chan = s_part + max(kThreads * V, a.C), *s_mean = s_chan + a.C;
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, blockIdx.x, r0, r1);
    if (b < 0) return;
    const int rows = int(r1 - r0);
    stage_rows<T, V>(s_x, x + r0 * a.C, rows, a.C, a.C);
    stage_wait();
    channel_sums<V, 1>(rows, a.C, s_part, s_chan, [&](int cv) {
        return [&, cv](int r, F2 (&acc)[1][kPairs<V>]) {
            const Vec<T, V> v = load_vec<T, V>(s_x + r * a.C + cv * V);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) acc[0][i] = acc[0][i] + pair_of(v, i);
        };
    });
    const float inv = 1.f / (float(rows) * float(a.per));
    group_sums(a.G, a.per, s_chan, [&](int g, float v) { s_mean[g] = v * inv; });
    __syncthreads();
    channel_sums<V, 1>(rows, a.C, s_part, s_chan, [&](int cv) {
        Channels<V> minus;
        minus.set(cv * V, a.per, [&](int, int g) { return -s_mean[g]; });
        return [&, cv, minus](int r, F2 (&acc)[1][kPairs<V>]) {
            const Vec<T, V> v = load_vec<T, V>(s_x + r * a.C + cv * V);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) {
                const F2 d = pair_of(v, i) + minus.v[i];
                acc[0][i] = fma2(d, d, acc[0][i]);
            }
        };
    });
    group_sums(a.G, a.per, s_chan, [&](int g, float v) {
        float* o = ws + (int64_t(blockIdx.x) * a.G + g) * 2;
        o[0] = s_mean[g];
        o[1] = v;
    });
}

// Forward, pass 2: Chan's merge of a graph's tiles, one block per (graph, group): each thread merges
// every 256th tile in order, then pairwise within warps and over the warps.
__global__ void __launch_bounds__(kThreads) norm_merge(NormArgs a, const float* __restrict__ ws) {
    __shared__ float s_w[3][kThreads / 32];
    const int64_t i = blockIdx.x;
    const int b = int(i / a.G), g = int(i % a.G);
    const int64_t r0 = a.offsets[b], n = a.offsets[b + 1] - r0;
    const int64_t t0 = r0 / a.R + b, tiles = (n + a.R - 1) / a.R;
    float cnt = 0.f, mean = 0.f, m2 = 0.f;
    auto merge = [&](float c2, float mean2, float m22) {
        if (c2 > 0.f) {
            const float tot = cnt + c2, d = mean2 - mean, w = c2 / tot;
            mean = fmaf(d, w, mean);
            m2 += m22 + d * d * cnt * w;
            cnt = tot;
        }
    };
    for (int64_t t = threadIdx.x; t < tiles; t += kThreads) {
        const float2 o = *reinterpret_cast<const float2*>(ws + ((t0 + t) * a.G + g) * 2);
        merge(float(min(int64_t(a.R), n - t * a.R)) * float(a.per), o.x, o.y);
    }
    auto lanes = [&](int from) {
        for (int k = from; k; k >>= 1) {
            const float c2 = __shfl_down_sync(0xffffffffu, cnt, k), u = __shfl_down_sync(0xffffffffu, mean, k),
                        w = __shfl_down_sync(0xffffffffu, m2, k);
            merge(c2, u, w);
        }
    };
    lanes(16);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (lane == 0) s_w[0][w] = cnt, s_w[1][w] = mean, s_w[2][w] = m2;
    __syncthreads();
    if (w > 0) return;
    const bool on = lane < kThreads / 32;
    cnt = on ? s_w[0][lane] : 0.f, mean = on ? s_w[1][lane] : 0.f, m2 = on ? s_w[2][lane] : 0.f;
    lanes(kThreads / 64);
    if (lane == 0) {
        a.mean[i] = mean;
        a.rstd[i] = rsqrtf((cnt > 0.f ? m2 / cnt : 0.f) + a.eps);
    }
}

// Forward, pass 3: y of a tile, the last tiles first.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_apply(NormArgs a, const T* __restrict__ x, T* __restrict__ y) {
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, gridDim.x - 1 - blockIdx.x, r0, r1);
    if (b < 0) return;
    const T* xt = x + r0 * a.C;
    T* yt = y + r0 * a.C;
    const int rows = int(r1 - r0);
    over_columns(
        a.C / V,
        [&](int cv, int rl, int par) {
            const int64_t g0 = int64_t(b) * a.G;
            Channels<V> minus, k, beta;
            minus.set(cv * V, a.per, [&](int, int g) { return -a.mean[g0 + g]; });
            k.set(cv * V, a.per, [&](int i, int g) { return a.rstd[g0 + g] * a.gamma[cv * V + i]; });
            beta.set(cv * V, a.per, [&](int i, int) { return a.beta[cv * V + i]; });
#pragma unroll 4
            for (int r = rl; r < rows; r += par) {
                const Vec<T, V> v = load_vec<T, V>(xt + int64_t(r) * a.C + cv * V);
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < kPairs<V>; ++i)
                    put_pair(o, i, act_of<ACT>(fma2(pair_of(v, i) + minus.v[i], k.v[i], beta.v[i])));
                store_vec<T, V>(yt + int64_t(r) * a.C + cv * V, o);
            }
        },
        [](int, int, int) {});
}

// Backward, pass 1: per-channel sums of dz and dz xh of each tile, ws[t][2][C].
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_bwd_tile_sums(NormArgs a, const T* __restrict__ x, const T* __restrict__ dy,
                                                               float* __restrict__ ws) {
    extern __shared__ __align__(16) float s_part[];  // [2 max(kThreads V, C)], then the sums [2 C]
    float* s_chan = s_part + 2 * max(kThreads * V, a.C);
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, blockIdx.x, r0, r1);
    if (b < 0) return;
    const T *xt = x + r0 * a.C, *gt = dy + r0 * a.C;
    channel_sums<V, 2>(int(r1 - r0), a.C, s_part, s_chan, [&](int cv) {
        const BwdChannel<V, ACT> ch(a, b, cv * V);
        return [&, cv, ch](int r, F2 (&acc)[2][kPairs<V>]) {
            const Vec<T, V> v = load_vec<T, V>(xt + int64_t(r) * a.C + cv * V), d = load_vec<T, V>(gt + int64_t(r) * a.C + cv * V);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) ch.add(pair_of(v, i), pair_of(d, i), i, acc[0][i], acc[1][i]);
        };
    });
    float* o = ws + int64_t(blockIdx.x) * 2 * a.C;
    for (int c = threadIdx.x; c < 2 * a.C; c += kThreads) o[c] = s_chan[c];
}

// Backward, pass 2: a graph's channel sums over its tiles to sums[b][2][C]: 32 channels a block, the
// warps share the tiles, then add in order.
__global__ void __launch_bounds__(kThreads) norm_bwd_merge(NormArgs a, const float* __restrict__ ws, float* __restrict__ sums) {
    __shared__ float s[kThreads / 32][32];
    const int per_graph = (2 * a.C + 31) / 32;
    const int b = int(blockIdx.x / per_graph), lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = int(blockIdx.x % per_graph) * 32 + lane;
    const int64_t r0 = a.offsets[b], n = a.offsets[b + 1] - r0;
    const int64_t t0 = r0 / a.R + b, tiles = (n + a.R - 1) / a.R;
    float acc = 0.f;
    if (c < 2 * a.C) {
#pragma unroll 4
        for (int64_t t = w; t < tiles; t += kThreads / 32) acc += ws[(t0 + t) * 2 * a.C + c];
    }
    s[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < 2 * a.C) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) t += s[k][lane];
        sums[int64_t(b) * 2 * a.C + c] = t;
    }
}

// Backward, pass 3: dx of a tile, the last tiles first.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_bwd_apply(NormArgs a, const T* __restrict__ x, const T* __restrict__ dy,
                                                           const float* __restrict__ sums, T* __restrict__ dx) {
    extern __shared__ __align__(16) float s_t[];  // gamma times the sums [2 C], then the groups' means [2 G]
    float *s_m1 = s_t + 2 * a.C, *s_m2 = s_m1 + a.G;
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, gridDim.x - 1 - blockIdx.x, r0, r1);
    if (b < 0) return;
    const float inv = 1.f / (float(a.offsets[b + 1] - a.offsets[b]) * float(a.per));
    for (int c = threadIdx.x; c < 2 * a.C; c += kThreads) s_t[c] = sums[int64_t(b) * 2 * a.C + c] * a.gamma[c < a.C ? c : c - a.C];
    __syncthreads();
    group_sums(a.G, a.per, s_t, [&](int g, float v) { s_m1[g] = v * inv; });
    group_sums(a.G, a.per, s_t + a.C, [&](int g, float v) { s_m2[g] = v * inv; });
    __syncthreads();
    const T *xt = x + r0 * a.C, *gt = dy + r0 * a.C;
    T* ot = dx + r0 * a.C;
    const int rows = int(r1 - r0);
    over_columns(
        a.C / V,
        [&](int cv, int rl, int par) {
            const BwdChannel<V, ACT> ch(a, b, cv * V);
            Channels<V> m1, m2;
            m1.set(cv * V, a.per, [&](int, int g) { return -s_m1[g]; });
            m2.set(cv * V, a.per, [&](int, int g) { return -s_m2[g]; });
#pragma unroll 2
            for (int r = rl; r < rows; r += par) {
                const Vec<T, V> v = load_vec<T, V>(xt + int64_t(r) * a.C + cv * V), d = load_vec<T, V>(gt + int64_t(r) * a.C + cv * V);
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < kPairs<V>; ++i) put_pair(o, i, ch.dx(pair_of(v, i), pair_of(d, i), i, m1.v[i], m2.v[i]));
                store_vec<T, V>(ot + int64_t(r) * a.C + cv * V, o);
            }
        },
        [](int, int, int) {});
}

// dgamma and dbeta: the graphs' channel sums added up, 32 of the 2 C sums a block; the warps share
// the graphs, then add in order.
__global__ void __launch_bounds__(1024) norm_bwd_params(int graphs, int C, const float* __restrict__ sums,
                                                        float* __restrict__ dgamma, float* __restrict__ dbeta) {
    __shared__ float s[32][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float acc = 0.f;
    if (c < 2 * C) {
#pragma unroll 8
        for (int b = w; b < graphs; b += 32) acc += sums[int64_t(b) * 2 * C + c];
    }
    s[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < 2 * C) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) t += s[k][lane];
        if (c < C)
            dbeta[c] = t;
        else
            dgamma[c - C] = t;
    }
}

// ------------------------------------------------------------------------------------ choice

size_t align256(size_t b) { return (b + 255) / 256 * 256; }
size_t elem_bytes(uvu_dtype t) { return t == UVU_F32 ? 4 : 2; }

// How a call is run.
struct Form {
    bool chip;
    int R;            // rows held by a block, or rows of a tile
    int slab, slabs;  // chip: channels of a block
    int K;            // chip: blocks of a cluster
    int64_t tiles;    // tiled
};

// The slab is the least run of whole groups of at least 128 bytes (a full line of each row).  The
// cluster is the smallest whose blocks hold the longest graph in kSmall bytes each (several blocks per
// SM overlap one another's phases), else in kLarge bytes; with fewer blocks than SMs it grows while
// a block keeps 64 rows.
Form form_of(const NormShape& s, bool bwd, int sms) {
    const size_t kSmall = bwd ? 56 << 10 : 40 << 10, kLarge = 160 << 10;
    const size_t e = elem_bytes(s.dtype), operands = bwd ? 2 : 1;
    const int V = int(16 / e), per = s.channels / s.groups;
    Form f = {};
    const int64_t unit = s.channels % V == 0 ? std::lcm(per, V) : per;
    const int64_t want = (int64_t(128 / e) + unit - 1) / unit * unit;
    f.slab = int(std::min<int64_t>(want, s.channels));
    f.slabs = (s.channels + f.slab - 1) / f.slab;
    const size_t row = size_t(f.slab) * e * operands;
    const int64_t blocks = int64_t(s.graphs) * f.slabs, longest = std::max<int64_t>(s.max_rows, 1);
    for (size_t room : {kSmall, kLarge}) {
        const int64_t R = int64_t(room / row), K = R > 0 ? (longest + R - 1) / R : 9;
        if (f.chip || K > 8) continue;
        f.chip = true;
        f.K = int(K);
        while (f.K < 8 && blocks * (f.K + 1) <= sms && longest >= 64 * (f.K + 1)) ++f.K;
        f.R = int((longest + f.K - 1) / f.K);
    }
    f.chip = f.chip && blocks * f.K < (int64_t(1) << 31);
    if (!f.chip) {
        f.R = int(std::min<size_t>(4096, std::max<size_t>(1, (32 << 10) / (size_t(s.channels) * e))));
        f.tiles = s.rows / f.R + s.graphs;
    }
    return f;
}

template <typename F>
cudaError_t allow_smem(F f, size_t bytes) {
    return bytes <= 48 << 10 ? cudaSuccess : cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

template <typename... P, typename... Q>
cudaError_t launch_cluster(void (*k)(P...), int64_t blocks, int K, size_t smem, cudaStream_t st, Q... args) {
    cudaError_t e = allow_smem(k, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(unsigned(blocks));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = unsigned(K);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k, static_cast<P>(args)...);
}

template <typename T, int V, int ACT>
cudaError_t fwd(NormArgs a, const Form& f, const T* x, T* y, float* ws, cudaStream_t st) {
    a.R = f.R, a.slab = f.slab, a.slabs = f.slabs;
    if (f.chip) {
        const size_t sm = (size_t(f.R) * f.slab * sizeof(T) + 15) / 16 * 16 +
                          (size_t(std::max(kThreads * V, f.slab)) + f.slab + 4 * (f.slab / a.per)) * 4;
        return launch_cluster(norm_fwd_chip<T, V, ACT>, int64_t(a.graphs) * f.slabs * f.K, f.K, sm, st, a, x, y);
    }
    const size_t sm = (size_t(f.R) * a.C * sizeof(T) + 15) / 16 * 16 + (size_t(std::max(kThreads * V, a.C)) + a.C + a.G) * 4;
    cudaError_t e = allow_smem(norm_tile_stats<T, V>, sm);
    if (e != cudaSuccess) return e;
    norm_tile_stats<T, V><<<unsigned(f.tiles), kThreads, sm, st>>>(a, x, ws);
    norm_merge<<<unsigned(int64_t(a.graphs) * a.G), kThreads, 0, st>>>(a, ws);
    norm_apply<T, V, ACT><<<unsigned(f.tiles), kThreads, 0, st>>>(a, x, y);
    return cudaGetLastError();
}

template <typename T, int V, int ACT>
cudaError_t bwd(NormArgs a, const Form& f, const T* x, const T* dy, T* dx, float* dgamma, float* dbeta, float* ws, cudaStream_t st) {
    a.R = f.R, a.slab = f.slab, a.slabs = f.slabs;
    float* sums = ws;
    cudaError_t e = cudaSuccess;
    if (f.chip) {
        const size_t sm = (size_t(f.R) * f.slab * sizeof(T) + 15) / 16 * 32 +
                          (2 * size_t(std::max(kThreads * V, f.slab)) + 4 * f.slab + 2 * (f.slab / a.per)) * 4;
        e = launch_cluster(norm_bwd_chip<T, V, ACT>, int64_t(a.graphs) * f.slabs * f.K, f.K, sm, st, a, x, dy, dx, sums);
    } else {
        float* tiles = ws + align256(size_t(a.graphs) * 2 * a.C * 4) / 4;
        const size_t sm = (size_t(std::max(kThreads * V, a.C)) * 2 + 2 * size_t(a.C)) * 4, sm3 = (2 * size_t(a.C) + 2 * size_t(a.G)) * 4;
        e = allow_smem(norm_bwd_tile_sums<T, V, ACT>, sm);
        if (e == cudaSuccess) e = allow_smem(norm_bwd_apply<T, V, ACT>, sm3);
        if (e != cudaSuccess) return e;
        norm_bwd_tile_sums<T, V, ACT><<<unsigned(f.tiles), kThreads, sm, st>>>(a, x, dy, tiles);
        norm_bwd_merge<<<unsigned(int64_t(a.graphs) * ((2 * a.C + 31) / 32)), kThreads, 0, st>>>(a, tiles, sums);
        norm_bwd_apply<T, V, ACT><<<unsigned(f.tiles), kThreads, sm3, st>>>(a, x, dy, sums, dx);
    }
    if (e != cudaSuccess) return e;
    norm_bwd_params<<<unsigned((2 * a.C + 31) / 32), 1024, 0, st>>>(a.graphs, a.C, sums, dgamma, dbeta);
    return cudaGetLastError();
}

// 16-byte vectors when every row begins on a 16-byte boundary, else single elements.
template <typename T, typename F>
cudaError_t by_vector(int C, uintptr_t any, F f) {
    if (C % int(16 / sizeof(T)) == 0 && (any & 15u) == 0) return f(std::integral_constant<int, int(16 / sizeof(T))>{});
    return f(std::integral_constant<int, 1>{});
}

template <typename T>
cudaError_t fwd_of(const NormArgs& a, const Form& f, uvu_act act, const void* x, void* y, void* ws, cudaStream_t st) {
    return by_vector<T>(a.C, reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y), [&](auto v) {
        constexpr int V = decltype(v)::value;
        const T* xp = static_cast<const T*>(x);
        T* yp = static_cast<T*>(y);
        float* w = static_cast<float*>(ws);
        return act == UVU_ACT_SILU ? fwd<T, V, UVU_ACT_SILU>(a, f, xp, yp, w, st) : fwd<T, V, UVU_ACT_NONE>(a, f, xp, yp, w, st);
    });
}
template <typename T>
cudaError_t bwd_of(const NormArgs& a, const Form& f, uvu_act act, const void* x, const void* dy, void* dx, float* dg, float* db,
                   void* ws, cudaStream_t st) {
    const uintptr_t any = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(dx);
    return by_vector<T>(a.C, any, [&](auto v) {
        constexpr int V = decltype(v)::value;
        const T *xp = static_cast<const T*>(x), *gp = static_cast<const T*>(dy);
        T* op = static_cast<T*>(dx);
        float* w = static_cast<float*>(ws);
        return act == UVU_ACT_SILU ? bwd<T, V, UVU_ACT_SILU>(a, f, xp, gp, op, dg, db, w, st)
                                   : bwd<T, V, UVU_ACT_NONE>(a, f, xp, gp, op, dg, db, w, st);
    });
}

NormArgs norm_args(const NormShape& s, const int32_t* offsets, const float* gamma, const float* beta, float* mean, float* rstd) {
    NormArgs a = {};
    a.rows = s.rows;
    a.graphs = s.graphs;
    a.C = s.channels;
    a.G = s.groups;
    a.per = s.channels / s.groups;
    a.eps = float(s.eps);
    a.offsets = offsets;
    a.gamma = gamma;
    a.beta = beta;
    a.mean = mean;
    a.rstd = rstd;
    return a;
}

}  // namespace

size_t norm_workspace(const NormShape& s, bool bwd, int sms) {
    const Form f = form_of(s, bwd, sms);
    if (!bwd) return f.chip ? 0 : size_t(f.tiles) * s.groups * 8;
    const size_t sums = size_t(s.graphs) * 2 * s.channels * 4;
    return f.chip ? sums : align256(sums) + size_t(f.tiles) * 2 * s.channels * 4;
}

cudaError_t launch_norm_fwd(const NormShape& s, const int32_t* offsets, const void* x, const float* gamma, const float* beta,
                            void* y, float* mean, float* rstd, void* ws, int sms, cudaStream_t st) {
    const NormArgs a = norm_args(s, offsets, gamma, beta, mean, rstd);
    const Form f = form_of(s, false, sms);
    switch (s.dtype) {
        case UVU_F32: return fwd_of<float>(a, f, s.act, x, y, ws, st);
        case UVU_BF16: return fwd_of<__nv_bfloat16>(a, f, s.act, x, y, ws, st);
        case UVU_F16: return fwd_of<__half>(a, f, s.act, x, y, ws, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_norm_bwd(const NormShape& s, const int32_t* offsets, const void* x, const void* dy, const float* gamma,
                            const float* beta, const float* mean, const float* rstd, void* dx, float* dgamma, float* dbeta,
                            void* ws, int sms, cudaStream_t st) {
    const NormArgs a = norm_args(s, offsets, gamma, beta, const_cast<float*>(mean), const_cast<float*>(rstd));
    const Form f = form_of(s, true, sms);
    switch (s.dtype) {
        case UVU_F32: return bwd_of<float>(a, f, s.act, x, dy, dx, dgamma, dbeta, ws, st);
        case UVU_BF16: return bwd_of<__nv_bfloat16>(a, f, s.act, x, dy, dx, dgamma, dbeta, ws, st);
        case UVU_F16: return bwd_of<__half>(a, f, s.act, x, dy, dx, dgamma, dbeta, ws, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace uvu
