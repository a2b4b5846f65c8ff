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
// Measured: 256 graphs of up to 1531 rows, 512 channels, bf16, forward and backward 393 us (2560 GB/s of the 1 GB
// that must move; the backward 258 us at 28% of DRAM's rate and 39% issue: the phases of a cluster - load, sums, exchange,
// write - follow one another, and three blocks an SM overlap them only in part); one graph of 200,001 rows, 256 channels,
// f16, 70 us (2920 GB/s).  Two rows in flight a thread and 256 threads a block were no faster.
#include <cooperative_groups.h>

#include <algorithm>
#include <cstdint>
#include <numeric>

#include "elem.h"
#include "plan.h"

namespace uvu {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 128, kMergeThreads = 256, kMaxCluster = 8;

// Division of values below 2^31 by a divisor that the host knows: n / d = (n m) >> (32 + s) with
// m = ceil(2^(32+s) / d), s = ceil(log2 d) - 1 (exact for n < 2^31: the error n (m d - 2^(32+s)) stays
// below 2^(32+s)).  An integer division costs some 25 instructions, which is what a short row's whole
// arithmetic costs.
struct Div {
    uint32_t d, m, s;
    static Div by(int d) {
        Div r = {uint32_t(d), 0, 0};
        while ((uint64_t(1) << (r.s + 1)) < r.d) ++r.s;
        r.m = uint32_t(((uint64_t(1) << (32 + r.s)) + r.d - 1) / r.d);  // d >= 2: below 2^32
        return r;
    }
    __device__ __forceinline__ int operator()(int n) const { return d == 1 ? n : int(__umulhi(uint32_t(n), m) >> s); }
};

struct NormArgs {
    int graphs, C, G, per;  // per = C / G
    Div by_per, by_slabs, by_size, by_lanes;
    int lanes, par, size;  // threads on a row, rows in parallel, blocks of a cluster
    int R;               // rows of a tile, or of a block's share that shared memory holds
    int slab, slabs;     // channels of a block (on-chip form), slabs of C
    float eps;
    const int32_t* offsets;
    const float *gamma, *beta;
    float *mean, *rstd;  // [B][G]
};

// The pairs of a vector; a single element is paired with zero.
template <int V>
constexpr int kPairs = V > 1 ? V / 2 : 1;
template <typename T, int V>
__device__ __forceinline__ F2 pair_of(const Vec<T, V>& v, int i) {
    if constexpr (V == 1)
        return F2(widen(v.v[0]), 0.f);
    else
        return F2(widen(v.v[2 * i]), widen(v.v[2 * i + 1]));
}
template <typename T, int V>
__device__ __forceinline__ void put_pair(Vec<T, V>& v, int i, F2 x) {
    const float2 b = x.both();
    if constexpr (V == 1) {
        v.v[0] = narrow<T>(b.x);
    } else if constexpr (sizeof(T) == 4) {
        v.v[2 * i] = b.x;
        v.v[2 * i + 1] = b.y;
    } else if constexpr (__is_same(T, __half)) {
        const __half2 h = __float22half2_rn(b);
        v.v[2 * i] = h.x, v.v[2 * i + 1] = h.y;
    } else {
        const __nv_bfloat162 h = __float22bfloat162_rn(b);
        v.v[2 * i] = h.x, v.v[2 * i + 1] = h.y;
    }
}

// 1 / (1 + exp(-z)): 2^x and 1/x to 2 ulp each; 2^x overflows to infinity where the sigmoid is below 2^-126, and 1/inf = 0.
__device__ __forceinline__ F2 sigmoid(F2 z) {
    float2 e = (z * F2(-1.4426950408889634f, -1.4426950408889634f)).both();
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    float2 d = (F2(e.x, e.y) + F2(1.f, 1.f)).both();
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(d.y));
    return F2(d.x, d.y);
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

// The block's threads over the vectors of a row of SC channels: consecutive threads take consecutive
// vectors, and `par` rows go in parallel.  Rows wider than the block take several rounds.
template <int V>
struct Columns {
    int vecs, lanes, par, rl, cl;  // vectors of a row, threads on a row, rows in parallel; the thread's row and vector
    // the last slab of a row may have fewer vectors than the lanes that the host chose
    __device__ __forceinline__ Columns(const NormArgs& a, int SC) : vecs(SC / V), lanes(a.lanes), par(a.par) {
        rl = a.by_lanes(threadIdx.x);
        cl = int(threadIdx.x) - rl * lanes;
    }
    // f(cv): the thread's vectors
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        if (rl < par)
            for (int cv = cl; cv < vecs; cv += lanes) f(cv);
    }
};

// Values per channel are kept in shared memory and read as the pairs of a thread's vector.
template <int V>
struct Channels {
    F2 v[kPairs<V>];
    __device__ __forceinline__ explicit Channels(const float* s) {  // 16-byte aligned where V > 1
        if constexpr (V == 1) {
            v[0] = F2(*s, 0.f);
        } else {
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const ulonglong2 q = reinterpret_cast<const ulonglong2*>(s)[i];
                v[2 * i].v = q.x, v[2 * i + 1].v = q.y;
            }
        }
    }
};
// f(c) for every channel c of `n`, shared out over the block.
template <typename F>
__device__ __forceinline__ void fill_channels(int n, F f) {
    for (int c = threadIdx.x; c < n; c += kThreads) f(c);
    __syncthreads();
}

// f(r, on_chip) for the thread's rows from r on: the first `held` are in shared memory (true_type), others in global memory.  Two loops,
// so that each has loads of its own kind.
template <int V, typename F>
__device__ __forceinline__ void each_row(const Columns<V>& co, int& r, int held, int rows, F f) {
#pragma unroll 1
    for (; r < held; r += co.par) f(r, std::true_type{});
#pragma unroll 1
    for (; r < rows; r += co.par) f(r, std::false_type{});
}
template <int V, typename F>
__device__ __forceinline__ void each_row(const Columns<V>& co, int held, int rows, F f) {
    int r = co.rl;
    each_row(co, r, held, rows, f);
}

constexpr int kRun = 1024;  // values that one thread adds up before it adds the sum to its others

// NS sums per channel over `rows` rows, to s_chan[s * SC + c].  f(cv) gives the function of (row, on_chip,
// acc) that adds a row's terms for vector cv.
template <int V, int NS, typename F>
__device__ __forceinline__ void channel_sums(const Columns<V>& co, int held, int rows, int SC, float* s_part, float* s_chan, F f) {
    const int width = co.lanes * V;
    for (int cv0 = 0; cv0 < co.vecs; cv0 += co.lanes) {
        const int n = min(co.lanes, co.vecs - cv0) * V;
        if (co.rl < co.par && cv0 + co.cl < co.vecs) {
            F2 acc[NS][kPairs<V>];
            auto clear = [&] {
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < kPairs<V>; ++i) acc[s][i] = F2(0.f, 0.f);
            };
            // to the thread's place, or to what it holds
            auto put = [&](bool more) {
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    float* o = s_part + (s * co.par + co.rl) * width + co.cl * V;
                    if constexpr (V == 1) {
                        *o = acc[s][0].both().x + (more ? *o : 0.f);
                    } else {
#pragma unroll
                        for (int i = 0; i < V / 4; ++i) {
                            float4* at = reinterpret_cast<float4*>(o) + i;
                            const float2 p = acc[s][2 * i].both(), q = acc[s][2 * i + 1].both();
                            const float4 old = more ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
                            *at = make_float4(p.x + old.x, p.y + old.y, q.x + old.z, q.y + old.w);
                        }
                    }
                }
            };
            clear();
            auto add = f(cv0 + co.cl);
            // A graph longer than promised: runs of kRun rows a thread, so that the sums' roundings do not grow with its length
            // (140,000 rows of 96 channels with max_rows = 1, bf16: rstd off by 5e-8, by 2e-5 in one run).
            const int64_t run = int64_t(kRun) * co.par;
            int r = co.rl;
            each_row(co, r, held, int(min(int64_t(rows), held + run)), [&](int i, auto on_chip) { add(i, on_chip, acc); });
            put(false);
#pragma unroll 1
            while (r < rows) {
                clear();
                each_row(co, r, 0, int(min(int64_t(rows), r + run)), [&](int i, auto on_chip) { add(i, on_chip, acc); });
                put(true);
            }
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < NS; ++s)
            for (int c = threadIdx.x; c < n; c += kThreads) {
                const float* p = s_part + s * co.par * width + c;
                float sum[2] = {0.f, 0.f};
                int k = 0;
#pragma unroll 4
                for (; k + 1 < co.par; k += 2) sum[0] += p[k * width], sum[1] += p[(k + 1) * width];
                if (k < co.par) sum[0] += p[k * width];
                s_chan[s * SC + cv0 * V + c] = sum[0] + sum[1];
            }
        __syncthreads();
    }
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
__device__ __forceinline__ void stage_rows(const Columns<V>& co, T* s, const T* x, int rows, int SC, int C) {
    co.each([&](int cv) {
        T* d = s + co.rl * SC + cv * V;
        const T* p = x + int64_t(co.rl) * C + cv * V;
        const int64_t step = int64_t(co.par) * C;
#pragma unroll 4
        for (int r = co.rl; r < rows; r += co.par, d += co.par * SC, p += step) stage_vec<T, V>(d, p);
    });
}
__device__ __forceinline__ void stage_wait() {
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
}

// ----------------------------------------------------------------------------------- on chip

struct Share {  // a block's part of a graph
    int b, c0, SC, rank, rows;
    int K;  // blocks that have rows (one, if none has); the others leave at once
    int n, each;  // rows of the graph, of a full share
    int64_t r0;
};
__device__ __forceinline__ Share share_of(const NormArgs& a) {
    Share s;
    const int id = a.by_size(blockIdx.x);
    s.rank = int(blockIdx.x) - id * a.size;
    s.b = a.by_slabs(id);
    s.c0 = (id - s.b * a.slabs) * a.slab;
    s.SC = min(a.slab, a.C - s.c0);
    const int first = a.offsets[s.b];
    s.n = a.offsets[s.b + 1] - first;
    // whole shares in rank order, so that short graphs need fewer blocks; a graph longer than max_rows
    // promised is shared out evenly
    const int each = s.n > a.R * a.size ? (s.n - 1) / a.size + 1 : a.R, lo = int(min(int64_t(s.n), int64_t(s.rank) * each));
    s.each = each;
    s.r0 = first + lo;
    s.rows = min(s.n - lo, each);
    s.K = s.n > each ? (s.n - 1) / each + 1 : 1;
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
            float v[kMaxCluster], s = 0.f;
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k) v[k] = k < K ? c.map_shared_rank(s_group, k)[i] : 0.f;
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k) s += v[k];
            s_sum[i] = s;
        }
    }
    __syncthreads();
}

// Mean and centred sum of squares of each group over the cluster, from the blocks' own (s_g: means,
// then sums of squares), merged in rank order.
__device__ __forceinline__ void cluster_merge(int groups, const Share& s, int per, float* s_g, float* s_mean, float* s_m2) {
    if (s.K == 1) {
        __syncthreads();
        for (int g = threadIdx.x; g < groups; g += kThreads) s_mean[g] = s_g[g], s_m2[g] = s_g[groups + g];
    } else {
        cg::cluster_group c = cg::this_cluster();
        __syncwarp();
        c.sync();
        for (int g = threadIdx.x; g < groups; g += kThreads) {
            float m[kMaxCluster], q[kMaxCluster];
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k)
                if (k < s.K) m[k] = c.map_shared_rank(s_g, k)[g], q[k] = c.map_shared_rank(s_g, k)[groups + g];
            float mean = m[0], m2 = q[0];
            int have = min(s.each, s.n);
#pragma unroll
            for (int k = 1; k < kMaxCluster; ++k)
                if (k < s.K) {
                    const int n = min(s.each, s.n - have);
                    const float d = m[k] - mean, w = float(n) / float(have + n);
                    mean = fmaf(d, w, mean);
                    m2 += q[k] + d * d * (float(have) * w) * float(per);
                    have += n;
                }
            s_mean[g] = mean;
            s_m2[g] = m2;
        }
    }
    __syncthreads();
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_fwd_chip(NormArgs a, const T* __restrict__ x, T* __restrict__ y) {
    extern __shared__ __align__(16) unsigned char smem[];
    const Share s = share_of(a);
    if (s.rank >= s.K) return;
    const Columns<V> co(a, s.SC);
    const int groups = a.by_per(s.SC), g0 = a.by_per(s.c0);
    T* s_x = reinterpret_cast<T*>(smem);
    float* s_part = reinterpret_cast<float*>(smem + (size_t(a.R) * a.slab * sizeof(T) + 15) / 16 * 16);
    const int pad = (a.slab + 3) & ~3;  // arrays per channel begin on 16 bytes
    float *s_chan = s_part + kThreads * V, *s_minus = s_chan + pad, *s_k = s_minus + pad, *s_beta = s_k + pad,
          *s_g = s_beta + pad, *s_mean = s_g + 2 * a.by_per(a.slab), *s_rstd = s_mean + a.by_per(a.slab);
    const T* xs = x + s.r0 * a.C + s.c0;
    const int held = min(s.rows, a.R);
    stage_rows<T, V>(co, s_x, xs, held, s.SC, a.C);
    stage_wait();
    auto row = [&](int r, int cv, auto on_chip) {
        if constexpr (decltype(on_chip)::value)
            return load_vec<T, V>(s_x + r * s.SC + cv * V);
        else
            return load_vec<T, V>(xs + int64_t(r) * a.C + cv * V);
    };
    channel_sums<V, 1>(co, held, s.rows, s.SC, s_part, s_chan, [&](int cv) {
        return [&, cv](int r, auto on_chip, F2 (&acc)[1][kPairs<V>]) {
            const Vec<T, V> v = row(r, cv, on_chip);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) acc[0][i] = acc[0][i] + pair_of(v, i);
        };
    });
    // the block's own mean and centred sum of squares per group, then Chan's merge over the cluster: one exchange
    const float own = s.rows > 0 ? 1.f / (float(s.rows) * float(a.per)) : 0.f;
    group_sums(groups, a.per, s_chan, [&](int g, float v) { s_g[g] = v * own; });
    __syncthreads();
    fill_channels(s.SC, [&](int c) { s_minus[c] = -s_g[a.by_per(c)]; });
    channel_sums<V, 1>(co, held, s.rows, s.SC, s_part, s_chan, [&](int cv) {
        const Channels<V> minus(s_minus + cv * V);
        return [&, cv, minus](int r, auto on_chip, F2 (&acc)[1][kPairs<V>]) {
            const Vec<T, V> v = row(r, cv, on_chip);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) {
                const F2 d = pair_of(v, i) + minus.v[i];
                acc[0][i] = fma2(d, d, acc[0][i]);
            }
        };
    });
    group_sums(groups, a.per, s_chan, [&](int g, float v) { s_g[groups + g] = v; });
    cluster_merge(groups, s, a.per, s_g, s_mean, s_rstd);
    if (s.K > 1) cg::this_cluster().barrier_arrive();  // the other blocks' sums have been read
    const float inv = s.n > 0 ? 1.f / (float(s.n) * float(a.per)) : 0.f;
    fill_channels(s.SC, [&](int c) {
        const int g = a.by_per(c);
        const float rstd = rsqrtf(s_rstd[g] * inv + a.eps);
        s_minus[c] = -s_mean[g];
        s_k[c] = rstd * a.gamma[s.c0 + c];
        s_beta[c] = a.beta[s.c0 + c];
        if (s.rank == 0 && c == g * a.per) {
            a.mean[int64_t(s.b) * a.G + g0 + g] = s_mean[g];
            a.rstd[int64_t(s.b) * a.G + g0 + g] = rstd;
        }
    });
    T* ys = y + s.r0 * a.C + s.c0;
    co.each([&](int cv) {
            const Channels<V> minus(s_minus + cv * V), k(s_k + cv * V), beta(s_beta + cv * V);
            each_row(co, held, s.rows, [&](int r, auto on_chip) {
                const Vec<T, V> v = row(r, cv, on_chip);
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < kPairs<V>; ++i)
                    put_pair(o, i, act_of<ACT>(fma2(pair_of(v, i) + minus.v[i], k.v[i], beta.v[i])));
                store_vec<T, V>(ys + int64_t(r) * a.C + cv * V, o);
            });
    });
    __syncwarp();
    if (s.K > 1) cg::this_cluster().barrier_wait();
}

// A thread's channels of the backward: xh and dz of a pair of values.
template <int V, int ACT>
struct BwdChannel {
    Channels<V> minus, rstd, gamma, beta;
    // s: the arrays that fill() wrote, of vector cv
    __device__ __forceinline__ BwdChannel(const float* s, int pad, int cv)
        : minus(s + cv * V), rstd(s + pad + cv * V), gamma(s + 2 * pad + cv * V), beta(s + 3 * pad + cv * V) {}
    static __device__ __forceinline__ void fill(const NormArgs& a, int b, int c0, int n, float* s, int pad) {
        fill_channels(n, [&](int c) {
            const int64_t g = int64_t(b) * a.G + a.by_per(c0 + c);
            s[c] = -a.mean[g];
            s[pad + c] = a.rstd[g];
            s[2 * pad + c] = a.gamma[c0 + c];
            s[3 * pad + c] = a.beta[c0 + c];
        });
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

// -mean(t) and -mean(t xh) of each channel's group, from the graph's channel sums.
__device__ __forceinline__ void group_means(const NormArgs& a, int n_channels, int64_t n, const float* sum0, const float* sum1,
                                            const float* s_gamma, float* s_m1, float* s_m2) {
    const float inv = n > 0 ? -1.f / (float(n) * float(a.per)) : 0.f;
    fill_channels(n_channels, [&](int c) { s_m1[c] = sum0[c] * s_gamma[c], s_m2[c] = sum1[c] * s_gamma[c]; });
    // a group's result replaces its first channel's value, which its own four lanes have read
    group_sums(a.by_per(n_channels), a.per, s_m1, [&](int g, float v) { s_m1[g * a.per] = v * inv; });
    group_sums(a.by_per(n_channels), a.per, s_m2, [&](int g, float v) { s_m2[g * a.per] = v * inv; });
    __syncthreads();
    fill_channels(n_channels, [&](int c) {
        const int g = a.by_per(c) * a.per;
        if (c != g) s_m1[c] = s_m1[g], s_m2[c] = s_m2[g];
    });
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_bwd_chip(NormArgs a, const T* __restrict__ x, const T* __restrict__ dy,
                                                          T* __restrict__ dx, float* __restrict__ sums) {
    extern __shared__ __align__(16) unsigned char smem[];
    const Share s = share_of(a);
    if (s.rank >= s.K) return;
    const Columns<V> co(a, s.SC);
    const size_t tile = (size_t(a.R) * a.slab * sizeof(T) + 15) / 16 * 16;
    T *s_x = reinterpret_cast<T*>(smem), *s_d = reinterpret_cast<T*>(smem + tile);
    float* s_part = reinterpret_cast<float*>(smem + 2 * tile);
    const int pad = (a.slab + 3) & ~3;  // arrays per channel begin on 16 bytes
    float *s_chan = s_part + 2 * kThreads * V, *s_sum = s_chan + 2 * pad, *s_ch = s_sum + 2 * pad, *s_m1 = s_ch + 4 * pad,
          *s_m2 = s_m1 + pad;
    const T *xs = x + s.r0 * a.C + s.c0, *ds = dy + s.r0 * a.C + s.c0;
    const int held = min(s.rows, a.R);
    stage_rows<T, V>(co, s_x, xs, held, s.SC, a.C);
    stage_rows<T, V>(co, s_d, ds, held, s.SC, a.C);
    BwdChannel<V, ACT>::fill(a, s.b, s.c0, s.SC, s_ch, pad);
    stage_wait();
    auto row = [&](const T* sm, const T* gm, int r, int cv, auto on_chip) {
        if constexpr (decltype(on_chip)::value)
            return load_vec<T, V>(sm + r * s.SC + cv * V);
        else
            return load_vec<T, V>(gm + int64_t(r) * a.C + cv * V);
    };
    channel_sums<V, 2>(co, held, s.rows, s.SC, s_part, s_chan, [&](int cv) {
        const BwdChannel<V, ACT> ch(s_ch, pad, cv);
        return [&, cv, ch](int r, auto on_chip, F2 (&acc)[2][kPairs<V>]) {
            const Vec<T, V> v = row(s_x, xs, r, cv, on_chip), d = row(s_d, ds, r, cv, on_chip);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) ch.add(pair_of(v, i), pair_of(d, i), i, acc[0][i], acc[1][i]);
        };
    });
    cluster_sums(2 * s.SC, s.K, s_chan, s_sum);
    if (s.K > 1) cg::this_cluster().barrier_arrive();  // the other blocks' sums have been read
    if (s.rank == 0)
        for (int c = threadIdx.x; c < 2 * s.SC; c += kThreads)
            sums[int64_t(s.b) * 2 * a.C + (c < s.SC ? s.c0 + c : a.C + s.c0 + c - s.SC)] = s_sum[c];
    group_means(a, s.SC, s.n, s_sum, s_sum + s.SC, s_ch + 2 * pad, s_m1, s_m2);
    T* os = dx + s.r0 * a.C + s.c0;
    co.each([&](int cv) {
            const BwdChannel<V, ACT> ch(s_ch, pad, cv);
            const Channels<V> m1(s_m1 + cv * V), m2(s_m2 + cv * V);
            each_row(co, held, s.rows, [&](int r, auto on_chip) {
                const Vec<T, V> v = row(s_x, xs, r, cv, on_chip), d = row(s_d, ds, r, cv, on_chip);
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < kPairs<V>; ++i) put_pair(o, i, ch.dx(pair_of(v, i), pair_of(d, i), i, m1.v[i], m2.v[i]));
                store_vec<T, V>(os + int64_t(r) * a.C + cv * V, o);
            });
    });
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
    const int pad = (a.C + 3) & ~3;  // arrays per channel begin on 16 bytes
    float *s_chan = s_part + kThreads * V, *s_minus = s_chan + pad, *s_mean = s_minus + pad;
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, blockIdx.x, r0, r1);
    if (b < 0) return;
    const int rows = int(r1 - r0);
    const Columns<V> co(a, a.C);
    stage_rows<T, V>(co, s_x, x + r0 * a.C, rows, a.C, a.C);
    stage_wait();
    channel_sums<V, 1>(co, rows, rows, a.C, s_part, s_chan, [&](int cv) {
        return [&, cv](int r, auto on_chip, F2 (&acc)[1][kPairs<V>]) {
            const Vec<T, V> v = load_vec<T, V>(s_x + r * a.C + cv * V);
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) acc[0][i] = acc[0][i] + pair_of(v, i);
        };
    });
    const float inv = 1.f / (float(rows) * float(a.per));
    group_sums(a.G, a.per, s_chan, [&](int g, float v) { s_mean[g] = v * inv; });
    __syncthreads();
    fill_channels(a.C, [&](int c) { s_minus[c] = -s_mean[a.by_per(c)]; });
    channel_sums<V, 1>(co, rows, rows, a.C, s_part, s_chan, [&](int cv) {
        const Channels<V> minus(s_minus + cv * V);
        return [&, cv, minus](int r, auto on_chip, F2 (&acc)[1][kPairs<V>]) {
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
// every kMergeThreads-th tile in order, then pairwise within warps and over the warps.
__global__ void __launch_bounds__(kMergeThreads) norm_merge(NormArgs a, const float* __restrict__ ws) {
    __shared__ float s_w[3][kMergeThreads / 32];
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
    // eight loads on their way together: a load and its merge in turn took 12 us of one graph's 72 at 3126 tiles
    constexpr int kAhead = 8;
    for (int64_t t = threadIdx.x; t < tiles; t += kAhead * kMergeThreads) {
        float2 o[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            o[k] = t + k * kMergeThreads < tiles ? *reinterpret_cast<const float2*>(ws + ((t0 + t + k * kMergeThreads) * a.G + g) * 2)
                                                 : make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            merge(float(max(int64_t(0), min(int64_t(a.R), n - (t + k * kMergeThreads) * a.R))) * float(a.per), o[k].x, o[k].y);
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
    const bool on = lane < kMergeThreads / 32;
    cnt = on ? s_w[0][lane] : 0.f, mean = on ? s_w[1][lane] : 0.f, m2 = on ? s_w[2][lane] : 0.f;
    lanes(kMergeThreads / 64);
    if (lane == 0) {
        a.mean[i] = mean;
        a.rstd[i] = rsqrtf((cnt > 0.f ? m2 / cnt : 0.f) + a.eps);
    }
}

// Forward, pass 3: y of a tile, the last tiles first.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_apply(NormArgs a, const T* __restrict__ x, T* __restrict__ y) {
    extern __shared__ __align__(16) float s_minus[];
    const int pad = (a.C + 3) & ~3;  // arrays per channel begin on 16 bytes
    float *s_k = s_minus + pad, *s_beta = s_k + pad;
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, gridDim.x - 1 - blockIdx.x, r0, r1);
    if (b < 0) return;
    const T* xt = x + r0 * a.C;
    T* yt = y + r0 * a.C;
    const int rows = int(r1 - r0);
    fill_channels(a.C, [&](int c) {
        const int64_t g = int64_t(b) * a.G + a.by_per(c);
        s_minus[c] = -a.mean[g];
        s_k[c] = a.rstd[g] * a.gamma[c];
        s_beta[c] = a.beta[c];
    });
    const Columns<V> co(a, a.C);
    co.each([&](int cv) {
            const Channels<V> minus(s_minus + cv * V), k(s_k + cv * V), beta(s_beta + cv * V);
#pragma unroll 4
            for (int r = co.rl; r < rows; r += co.par) {
                const Vec<T, V> v = load_vec<T, V>(xt + int64_t(r) * a.C + cv * V);
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < kPairs<V>; ++i)
                    put_pair(o, i, act_of<ACT>(fma2(pair_of(v, i) + minus.v[i], k.v[i], beta.v[i])));
                store_vec<T, V>(yt + int64_t(r) * a.C + cv * V, o);
            }
    });
}

// Backward, pass 1: per-channel sums of dz and dz xh of each tile, ws[t][2][C].
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_bwd_tile_sums(NormArgs a, const T* __restrict__ x, const T* __restrict__ dy,
                                                               float* __restrict__ ws) {
    extern __shared__ __align__(16) float s_part[];  // [2 kThreads V], the sums [2 pad], the channels [4 pad]
    const int pad = (a.C + 3) & ~3;                   // arrays per channel begin on 16 bytes
    float *s_chan = s_part + 2 * kThreads * V, *s_ch = s_chan + 2 * pad;
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, blockIdx.x, r0, r1);
    if (b < 0) return;
    const T *xt = x + r0 * a.C, *gt = dy + r0 * a.C;
    BwdChannel<V, ACT>::fill(a, b, 0, a.C, s_ch, pad);
    const Columns<V> co(a, a.C);
    channel_sums<V, 2>(co, 0, int(r1 - r0), a.C, s_part, s_chan, [&](int cv) {
        const BwdChannel<V, ACT> ch(s_ch, pad, cv);
        return [&, cv, ch](int r, auto on_chip, F2 (&acc)[2][kPairs<V>]) {
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
__global__ void __launch_bounds__(kMergeThreads) norm_bwd_merge(NormArgs a, const float* __restrict__ ws, float* __restrict__ sums) {
    __shared__ float s[kMergeThreads / 32][32];
    const int per_graph = (2 * a.C + 31) / 32;
    const int b = int(blockIdx.x / per_graph), lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = int(blockIdx.x % per_graph) * 32 + lane;
    const int64_t r0 = a.offsets[b], n = a.offsets[b + 1] - r0;
    const int64_t t0 = r0 / a.R + b, tiles = (n + a.R - 1) / a.R;
    float acc = 0.f;
    if (c < 2 * a.C) {
        for (int64_t t = w; t < tiles;) {
            float run = 0.f;
            const int64_t end = min(tiles, t + kRun * (kMergeThreads / 32));
#pragma unroll 4
            for (; t < end; t += kMergeThreads / 32) run += ws[(t0 + t) * 2 * a.C + c];
            acc += run;
        }
    }
    s[w][lane] = acc;
    __syncthreads();
    if (w == 0 && c < 2 * a.C) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kMergeThreads / 32; ++k) t += s[k][lane];
        sums[int64_t(b) * 2 * a.C + c] = t;
    }
}

// Backward, pass 3: dx of a tile, the last tiles first.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) norm_bwd_apply(NormArgs a, const T* __restrict__ x, const T* __restrict__ dy,
                                                           const float* __restrict__ sums, T* __restrict__ dx) {
    extern __shared__ __align__(16) float s_ch[];  // the channels [4 pad], the means of t and t xh per channel [2 pad]
    const int pad = (a.C + 3) & ~3;                // arrays per channel begin on 16 bytes
    float *s_m1 = s_ch + 4 * pad, *s_m2 = s_m1 + pad;
    int64_t r0, r1;
    const int b = tile_graph(a.offsets, a.graphs, a.R, gridDim.x - 1 - blockIdx.x, r0, r1);
    if (b < 0) return;
    BwdChannel<V, ACT>::fill(a, b, 0, a.C, s_ch, pad);
    const float* sum = sums + int64_t(b) * 2 * a.C;
    group_means(a, a.C, a.offsets[b + 1] - a.offsets[b], sum, sum + a.C, s_ch + 2 * pad, s_m1, s_m2);
    const T *xt = x + r0 * a.C, *gt = dy + r0 * a.C;
    T* ot = dx + r0 * a.C;
    const int rows = int(r1 - r0);
    const Columns<V> co(a, a.C);
    co.each([&](int cv) {
            const BwdChannel<V, ACT> ch(s_ch, pad, cv);
            const Channels<V> m1(s_m1 + cv * V), m2(s_m2 + cv * V);
#pragma unroll 2
            for (int r = co.rl; r < rows; r += co.par) {
                const Vec<T, V> v = load_vec<T, V>(xt + int64_t(r) * a.C + cv * V), d = load_vec<T, V>(gt + int64_t(r) * a.C + cv * V);
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < kPairs<V>; ++i) put_pair(o, i, ch.dx(pair_of(v, i), pair_of(d, i), i, m1.v[i], m2.v[i]));
                store_vec<T, V>(ot + int64_t(r) * a.C + cv * V, o);
            }
    });
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
        for (int b = w; b < graphs;) {
            float run = 0.f;
            const int end = min(graphs, b + kRun * 32);
#pragma unroll 8
            for (; b < end; b += 32) run += sums[int64_t(b) * 2 * C + c];
            acc += run;
        }
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

size_t elem_bytes(uvu_dtype t) { return t == UVU_F32 ? 4 : 2; }

// How a call is run.
struct Form {
    bool chip;
    int R;            // rows held by a block, or rows of a tile
    int slab, slabs;  // chip: channels of a block
    int K;            // chip: blocks of a cluster
    int64_t tiles;    // tiled
};

// Shared memory of a block of the on-chip form beside its rows.
size_t chip_fixed(bool bwd, int slab, int per, int V) {
    const size_t pad = (size_t(slab) + 3) & ~size_t(3);
    return 32 + (bwd ? 2 * size_t(kThreads) * V + 10 * pad : size_t(kThreads) * V + 4 * pad + 4 * size_t(slab / per)) * 4;
}

// On chip where the longest graph fits: 393 against 504 us (forward and backward, 256 graphs of up to 1531 rows, 512
// channels, bf16), 14 against 37 (64 of up to 127, 128 channels, fp32).  The slab is the least run of whole groups of at least 128 bytes (a full line of each row).  The
// cluster is the smallest whose blocks hold the longest graph, several blocks to an SM if possible (they
// overlap one another's phases); with fewer blocks than SMs it grows while a block keeps 64 rows (one graph of 1000
// rows: 15.3 against 18.7 us, both ways).
Form form_of(const NormShape& s, bool bwd, int sms) {
    const size_t e = elem_bytes(s.dtype);
    const int V = int(16 / e), per = s.channels / s.groups;
    // shared memory of a block: four (backward: three, its registers' limit) per SM, or one
    const size_t rooms[2] = {size_t(bwd ? 74 : 56) << 10, size_t(224) << 10};
    Form f = {};
    const int64_t unit = s.channels % V == 0 ? std::lcm(per, V) : per;
    const int64_t want = (int64_t(128 / e) + unit - 1) / unit * unit;
    f.slab = int(std::min<int64_t>(want, s.channels));
    f.slabs = (s.channels + f.slab - 1) / f.slab;
    const size_t row = size_t(f.slab) * e * (bwd ? 2 : 1), fixed = chip_fixed(bwd, f.slab, per, V);
    const int64_t blocks = int64_t(s.graphs) * f.slabs, longest = std::max<int64_t>(s.max_rows, 1);
    for (size_t room : rooms) {
        const int64_t R = room > fixed ? int64_t((room - fixed) / row) : 0, K = R > 0 ? (longest + R - 1) / R : kMaxCluster + 1;
        if (f.chip || K > kMaxCluster) continue;
        f.chip = true;
        f.K = int(K);
        while (f.K < kMaxCluster && blocks * (f.K + 1) <= sms && longest >= 64 * (f.K + 1)) ++f.K;
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
    return bytes <= 48 << 10 ? cudaSuccess : allow_most_smem(f, bytes);
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

void set_form(NormArgs& a, const Form& f, int V) {
    a.R = f.R, a.slab = f.slab, a.slabs = f.slabs, a.size = f.chip ? f.K : 1;
    a.lanes = std::min((f.chip ? f.slab : a.C) / V, kThreads);
    a.par = kThreads / a.lanes;
    a.by_per = Div::by(a.per), a.by_slabs = Div::by(std::max(a.slabs, 1)), a.by_size = Div::by(a.size), a.by_lanes = Div::by(a.lanes);
}

template <typename T, int V, int ACT>
cudaError_t fwd(NormArgs a, const Form& f, const T* x, T* y, float* ws, cudaStream_t st) {
    set_form(a, f, V);
    if (f.chip) {
        const size_t sm = (size_t(f.R) * f.slab * sizeof(T) + 15) / 16 * 16 + chip_fixed(false, f.slab, a.per, V);
        return launch_cluster(norm_fwd_chip<T, V, ACT>, int64_t(a.graphs) * f.slabs * f.K, f.K, sm, st, a, x, y);
    }
    const int pad = (a.C + 3) & ~3;
    const size_t sm = (size_t(f.R) * a.C * sizeof(T) + 15) / 16 * 16 + (size_t(kThreads) * V + 2 * pad + a.G) * 4,
                 sm3 = size_t(pad) * 12;
    cudaError_t e = allow_smem(norm_tile_stats<T, V>, sm);
    if (e == cudaSuccess) e = allow_smem(norm_apply<T, V, ACT>, sm3);
    if (e != cudaSuccess) return e;
    norm_tile_stats<T, V><<<unsigned(f.tiles), kThreads, sm, st>>>(a, x, ws);
    norm_merge<<<unsigned(int64_t(a.graphs) * a.G), kMergeThreads, 0, st>>>(a, ws);
    norm_apply<T, V, ACT><<<unsigned(f.tiles), kThreads, sm3, st>>>(a, x, y);
    return cudaGetLastError();
}

template <typename T, int V, int ACT>
cudaError_t bwd(NormArgs a, const Form& f, const T* x, const T* dy, T* dx, float* dgamma, float* dbeta, float* ws, cudaStream_t st) {
    set_form(a, f, V);
    float* sums = ws;
    cudaError_t e = cudaSuccess;
    if (f.chip) {
        const size_t sm = (size_t(f.R) * f.slab * sizeof(T) + 15) / 16 * 32 + chip_fixed(true, f.slab, a.per, V);
        e = launch_cluster(norm_bwd_chip<T, V, ACT>, int64_t(a.graphs) * f.slabs * f.K, f.K, sm, st, a, x, dy, dx, sums);
    } else {
        float* tiles = ws + align256(size_t(a.graphs) * 2 * a.C * 4) / 4;
        const int pad = (a.C + 3) & ~3;
        const size_t sm = (2 * size_t(kThreads) * V + 6 * size_t(pad)) * 4, sm3 = 6 * size_t(pad) * 4;
        e = allow_smem(norm_bwd_tile_sums<T, V, ACT>, sm);
        if (e == cudaSuccess) e = allow_smem(norm_bwd_apply<T, V, ACT>, sm3);
        if (e != cudaSuccess) return e;
        norm_bwd_tile_sums<T, V, ACT><<<unsigned(f.tiles), kThreads, sm, st>>>(a, x, dy, tiles);
        norm_bwd_merge<<<unsigned(int64_t(a.graphs) * ((2 * a.C + 31) / 32)), kMergeThreads, 0, st>>>(a, tiles, sums);
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
