// Attention of a graph's nodes to another set of states, over a packed batch of graphs.
//
// For graph b, head h and the kv head h / group, over the kept states j of the graph:
//     S_ij = scale q_i . k_j,  lse_i = log sum_j exp S_ij,  P_ij = exp(S_ij - lse_i),  o_i = sum_j P_ij v_j
// A row without a kept state gets o = 0, lse = -inf and takes part in no gradient.  Backward, with
// delta_i = do_i . o_i (= sum_j P_ij dP_ij):
//     dP = do v^T,  dS = P (dP - delta),  dq = scale dS k,  dk = scale dS^T q,  dv = P^T do,
// dk and dv summed over the heads of the group.  Nothing of size rows x states is stored: the
// forward keeps a running maximum and sum per row, the backward recomputes P from lse.
//
// Values of masked states are never used: their rows are read as zeros and their S is -inf, so
// infinities and NaN there change nothing.
//
// This file holds the launch choices and the CUDA-core kernels: 64 x 64 tiles, operands widened
// to fp32 in shared memory, 256 threads with 4 x 4 scores each.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "elem.h"

namespace uvu {
namespace {

constexpr int kThreads = 256;
constexpr int kT = 64;       // rows and states of a tile
constexpr int kSP = kT + 4;  // pitch of a score tile

// Rows r0 .. r0 + 64 of a [rows][heads][D] operand to shared memory [64][DP + 4]; rows at or past
// `rows`, columns past D and rows that `use` refuses are zeros.  `at(r)` gives a row's address.
template <typename T, int DP, typename At, typename Use>
__device__ __forceinline__ void load_tile(float* s, int D, At at, Use use) {
    constexpr int P = DP + 4;
    for (int e = threadIdx.x; e < kT * DP; e += kThreads) {
        const int r = e / DP, d = e % DP;
        s[r * P + d] = d < D && use(r) ? widen(at(r)[d]) : 0.f;
    }
}

// acc[i][j] += sum_d a[row ty*4+i][d] b[row tx+16 j][d]
template <int DP>
__device__ __forceinline__ void dot_tile(const float* a, const float* b, int ty, int tx, float (&acc)[4][4]) {
    constexpr int P = DP + 4;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ty * 4 + i) * P + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * P + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] += x[i].x * y[j].x + x[i].y * y[j].y + x[i].z * y[j].z + x[i].w * y[j].w;
    }
}

// acc[i][c] += sum_k p[ty*4+i][k] b[k][tx + 16 c]   (TRANS: p[k][ty*4+i])
template <int DP, bool TRANS>
__device__ __forceinline__ void mul_tile(const float* p, const float* b, int ty, int tx, float (&acc)[4][DP / 16]) {
    constexpr int P = DP + 4;
    for (int k = 0; k < kT; ++k) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = TRANS ? p[k * kSP + ty * 4 + i] : p[(ty * 4 + i) * kSP + k];
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const float y = b[k * P + tx + 16 * c];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i][c] = fmaf(x[i], y, acc[i][c]);
        }
    }
}

struct Range {
    int64_t lo, hi;
};
// The part of n values that split s of `splits` takes, whole tiles of R.
__device__ __forceinline__ Range split_range(int64_t n, int s, int splits, int R) {
    const int64_t tiles = (n + R - 1) / R, per = (tiles + splits - 1) / splits;
    return {min(n, s * per * R), min(n, (s + 1) * per * R)};
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attn_fwd_simple(AttnArgs a) {
    extern __shared__ __align__(16) float smem[];
    constexpr int P = DP + 4;
    float *sq = smem, *sk = sq + kT * P, *sv = sk + kT * P, *sp = sv + kT * P;
    __shared__ uint8_t s_keep[kT];
    const AttnTile tl = attn_tile(a.q_off, a.graphs, a.group, kT, blockIdx.x);
    if (tl.graph < 0) return;
    const int h = blockIdx.y, split = blockIdx.z;
    const int64_t q0 = a.q_off[tl.graph], k0 = a.k_off[tl.graph], nk = a.k_off[tl.graph + 1] - k0;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    auto qrow = [&](int64_t r) { return q0 + r / a.group; };
    auto qhead = [&](int64_t r) { return int64_t(h) * a.group + r % a.group; };
    load_tile<T, DP>(
        sq, a.D,
        [&](int r) {
            const int64_t p = tl.row0 + r;
            return static_cast<const T*>(a.q) + qrow(p) * a.q_row + qhead(p) * a.q_head;
        },
        [&](int r) { return tl.row0 + r < tl.rows; });
    float m[4], l[4], o[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) o[i][c] = 0.f;
    }
    const Range kr = split_range(nk, split, a.splits, kT);
    for (int64_t kb = kr.lo; kb < kr.hi; kb += kT) {
        __syncthreads();
        if (threadIdx.x < kT) {
            const int64_t j = kb + threadIdx.x;
            s_keep[threadIdx.x] = j < kr.hi && (!a.keep || a.keep[k0 + j]);
        }
        __syncthreads();
        load_tile<T, DP>(
            sk, a.D, [&](int r) { return static_cast<const T*>(a.k) + (k0 + kb + r) * a.k_row + h * a.k_head; },
            [&](int r) { return s_keep[r] != 0; });
        load_tile<T, DP>(
            sv, a.D, [&](int r) { return static_cast<const T*>(a.v) + (k0 + kb + r) * a.v_row + h * a.v_head; },
            [&](int r) { return s_keep[r] != 0; });
        __syncthreads();
        float s[4][4] = {};
        dot_tile<DP>(sq, sk, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = s_keep[tx + 16 * j] ? s[i][j] * a.scale_log2 : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int k = 8; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
            const float mn = fmaxf(m[i], top), base = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m[i] - base);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(s[i][j] - base);
                sp[(ty * 4 + i) * kSP + tx + 16 * j] = p;
                sum += p;
            }
            l[i] = l[i] * f + sum;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) o[i][c] *= f;
        }
        __syncthreads();
        mul_tile<DP, false>(sp, sv, ty, tx, o);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float sum = l[i];
#pragma unroll
        for (int k = 8; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        const int64_t p = tl.row0 + ty * 4 + i;
        if (p >= tl.rows) continue;
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        const float lse = sum == 0.f ? -INFINITY : (m[i] + log2f(sum)) * 0.6931471805599453f;
        const int64_t row = qrow(p), head = qhead(p);
        if (a.splits > 1) {
            const int64_t at = (int64_t(split) * a.nq + row) * a.Hq + head;
            if (tx == 0) a.part_lse[at] = lse;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c)
                if (tx + 16 * c < a.D) a.part_o[at * a.D + tx + 16 * c] = o[i][c] * inv;
        } else {
            if (tx == 0) a.lse[row * a.Hq + head] = lse;
            T* po = static_cast<T*>(a.out) + row * a.o_row + head * a.o_head;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c)
                if (tx + 16 * c < a.D) po[tx + 16 * c] = narrow<T>(o[i][c] * inv);
        }
    }
}

// Joins the splits of a row: o = sum_s exp(lse_s - lse) o_s.  One warp per (row, head).
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_fwd_join(AttnArgs a) {
    const int64_t rh = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t total = a.nq * a.Hq;
    if (rh >= total) return;
    float top = -INFINITY;
    for (int s = lane; s < a.splits; s += 32) top = fmaxf(top, a.part_lse[s * total + rh]);
#pragma unroll
    for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    float sum = 0.f;
    for (int s = lane; s < a.splits; s += 32) {
        const float x = a.part_lse[s * total + rh];
        sum += x == -INFINITY ? 0.f : expf(x - top);
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    const float lse = sum == 0.f ? -INFINITY : top + logf(sum);
    if (lane == 0) a.lse[rh] = lse;
    T* po = static_cast<T*>(a.out) + (rh / a.Hq) * a.o_row + (rh % a.Hq) * a.o_head;
    for (int d = lane; d < a.D; d += 32) {
        float o = 0.f;
        for (int s = 0; s < a.splits; ++s) {
            const float x = a.part_lse[s * total + rh];
            if (x != -INFINITY) o = fmaf(expf(x - lse), a.part_o[(s * total + rh) * a.D + d], o);
        }
        po[d] = narrow<T>(o);
    }
}

// delta[row][head] = sum_d d_out out.  One warp per (row, head).
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_delta(AttnArgs a) {
    const int64_t rh = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (rh >= a.nq * a.Hq) return;
    const int64_t at = (rh / a.Hq) * a.o_row + (rh % a.Hq) * a.o_head;
    float s = 0.f;
    for (int d = lane; d < a.D; d += 32)
        s = fmaf(widen(static_cast<const T*>(a.d_out)[at + d]), widen(static_cast<const T*>(a.out)[at + d]), s);
#pragma unroll
    for (int k = 16; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0) a.delta[rh] = s;
}

// The backward's P and dS of one (row tile, state tile) pair into sp and sds.
template <int DP>
__device__ __forceinline__ void bwd_scores(const AttnArgs& a, const float* sq, const float* sk, const float* sv, const float* sdo,
                                           const float* s_lse, const float* s_delta, const uint8_t* s_keep, int ty, int tx,
                                           float* sp, float* sds) {
    float s[4][4] = {}, dp[4][4] = {};
    dot_tile<DP>(sq, sk, ty, tx, s);
    dot_tile<DP>(sdo, sv, ty, tx, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lse = s_lse[ty * 4 + i], delta = s_delta[ty * 4 + i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool on = s_keep[tx + 16 * j] && lse != -INFINITY;
            const float p = on ? exp2f(s[i][j] * a.scale_log2 - lse * 1.4426950408889634f) : 0.f;
            sp[(ty * 4 + i) * kSP + tx + 16 * j] = p;
            sds[(ty * 4 + i) * kSP + tx + 16 * j] = on ? p * (dp[i][j] - delta) * a.scale : 0.f;
        }
    }
}

// dq (KV == false): a row tile over the states.  dk, dv (KV == true): a state tile over the rows.
template <typename T, int DP, bool KV>
__global__ void __launch_bounds__(kThreads) attn_bwd_simple(AttnArgs a) {
    extern __shared__ __align__(16) float smem[];
    constexpr int P = DP + 4;
    float *sq = smem, *sk = sq + kT * P, *sv = sk + kT * P, *sdo = sv + kT * P, *sp = sdo + kT * P, *sds = sp + kT * kSP;
    __shared__ float s_lse[kT], s_delta[kT];
    __shared__ uint8_t s_keep[kT];
    const AttnTile tl = KV ? attn_tile(a.k_off, a.graphs, 1, kT, blockIdx.x) : attn_tile(a.q_off, a.graphs, a.group, kT, blockIdx.x);
    if (tl.graph < 0) return;
    const int h = blockIdx.y, split = blockIdx.z;
    const int64_t q0 = a.q_off[tl.graph], k0 = a.k_off[tl.graph];
    const int64_t rows = (a.q_off[tl.graph + 1] - q0) * a.group, nk = a.k_off[tl.graph + 1] - k0;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    auto load_rows = [&](int64_t r0) {
        auto use = [&](int r) { return r0 + r < rows; };
        load_tile<T, DP>(
            sq, a.D,
            [&](int r) {
                const int64_t p = r0 + r;
                return static_cast<const T*>(a.q) + (q0 + p / a.group) * a.q_row + (int64_t(h) * a.group + p % a.group) * a.q_head;
            },
            use);
        load_tile<T, DP>(
            sdo, a.D,
            [&](int r) {
                const int64_t p = r0 + r;
                return static_cast<const T*>(a.d_out) + (q0 + p / a.group) * a.o_row +
                       (int64_t(h) * a.group + p % a.group) * a.o_head;
            },
            use);
        if (threadIdx.x < kT) {
            const int64_t p = r0 + threadIdx.x;
            const int64_t at = (q0 + p / a.group) * a.Hq + int64_t(h) * a.group + p % a.group;
            s_lse[threadIdx.x] = p < rows ? a.lse[at] : -INFINITY;
            s_delta[threadIdx.x] = p < rows ? a.delta[at] : 0.f;
        }
    };
    auto load_states = [&](int64_t kb) {
        if (threadIdx.x < kT) {
            const int64_t j = kb + threadIdx.x;
            s_keep[threadIdx.x] = j < nk && (!a.keep || a.keep[k0 + j]);
        }
        __syncthreads();
        auto use = [&](int r) { return s_keep[r] != 0; };
        load_tile<T, DP>(
            sk, a.D, [&](int r) { return static_cast<const T*>(a.k) + (k0 + kb + r) * a.k_row + h * a.k_head; }, use);
        load_tile<T, DP>(
            sv, a.D, [&](int r) { return static_cast<const T*>(a.v) + (k0 + kb + r) * a.v_row + h * a.v_head; }, use);
    };
    float g1[4][DP / 16], g2[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) g1[i][c] = g2[i][c] = 0.f;
    if constexpr (KV) {
        load_states(tl.row0);
        const Range rr = split_range(rows, split, a.splits, kT);
        for (int64_t r0 = rr.lo; r0 < rr.hi; r0 += kT) {
            __syncthreads();
            load_rows(r0);
            __syncthreads();
            bwd_scores<DP>(a, sq, sk, sv, sdo, s_lse, s_delta, s_keep, ty, tx, sp, sds);
            __syncthreads();
            mul_tile<DP, true>(sds, sq, ty, tx, g1);
            mul_tile<DP, true>(sp, sdo, ty, tx, g2);
        }
    } else {
        load_rows(tl.row0);
        const Range kr = split_range(nk, split, a.splits, kT);
        for (int64_t kb = kr.lo; kb < kr.hi; kb += kT) {
            __syncthreads();
            load_states(kb);
            __syncthreads();
            bwd_scores<DP>(a, sq, sk, sv, sdo, s_lse, s_delta, s_keep, ty, tx, sp, sds);
            __syncthreads();
            mul_tile<DP, false>(sds, sk, ty, tx, g1);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t p = tl.row0 + ty * 4 + i;
        if (p >= tl.rows) continue;
        const int64_t at = KV ? (k0 + p) * a.Hkv + h : (q0 + p / a.group) * a.Hq + int64_t(h) * a.group + p % a.group;
        const int64_t n = KV ? a.nk * a.Hkv : a.nq * a.Hq;  // (row, head) pairs of the gradient
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) {
            const int d = tx + 16 * c;
            if (d >= a.D) continue;
            if (a.splits > 1) {
                a.part_o[(split * n + at) * a.D + d] = g1[i][c];
                if (KV) a.part_o[((int64_t(a.splits) + split) * n + at) * a.D + d] = g2[i][c];
            } else {
                static_cast<T*>(KV ? a.dk : a.dq)[at * a.D + d] = narrow<T>(g1[i][c]);
                if (KV) static_cast<T*>(a.dv)[at * a.D + d] = narrow<T>(g2[i][c]);
            }
        }
    }
}

// dst[i] = sum_s part[s][i], in the order of the splits.
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_bwd_join(int64_t n, int splits, const float* __restrict__ part, T* __restrict__ dst) {
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
    for (int k = 0; k < splits; ++k) s += part[k * n + i];
    dst[i] = narrow<T>(s);
}

// Splits of the inner axis: as many as fill the card's SMs once, when there are fewer tiles than
// SMs, but no piece shorter than four tiles.
int splits_for(int64_t tiles, int64_t inner, int R, int sms) {
    if (tiles <= 0 || tiles >= sms) return 1;
    const int64_t want = (sms + tiles - 1) / tiles, most = std::max<int64_t>(1, inner / (4 * R));
    return int(std::min<int64_t>(std::min(want, most), 64));
}

int64_t row_tiles(const AttnShape& s, int R) { return s.n_q * (s.q_heads / s.kv_heads) / R + s.n_graphs; }
int64_t state_tiles(const AttnShape& s, int R) { return s.n_k / R + s.n_graphs; }

enum class Engine { kCuda, kMma, kPlanes };
struct Choice {
    Engine engine;
    int nt;             // row tiles of 128 per block of the 16-bit forward
    int R;              // rows or states of a tile
    int64_t fwd_tiles;  // tile numbers of the forward
    int fwd, dq, dkv;   // splits
};
Choice choose(const AttnShape& s, int sms) {
    const int64_t group = s.q_heads / s.kv_heads;
    // tiles that have work, at most
    const auto rows_busy = [&](int R) {
        return std::min(row_tiles(s, R), int64_t(s.n_graphs) * ((s.max_q * group + R - 1) / R)) * s.kv_heads;
    };
    const auto states_busy = [&](int R) {
        return std::min(state_tiles(s, R), int64_t(s.n_graphs) * ((s.max_k + R - 1) / R)) * s.kv_heads;
    };
    Choice c;
    c.engine = s.dtype != UVU_F32 ? Engine::kMma : s.head_dim <= kPlaneDim ? Engine::kPlanes : Engine::kCuda;
    c.R = c.engine == Engine::kCuda ? kT : 128;
    c.nt = c.engine == Engine::kMma && rows_busy(256) >= sms && s.max_q * group > 128 ? 2 : 1;
    c.fwd_tiles = row_tiles(s, c.R * c.nt);
    c.fwd = splits_for(rows_busy(c.R * c.nt), s.max_k, c.R, sms);
    c.dq = splits_for(rows_busy(c.R), s.max_k, c.R, sms);
    c.dkv = splits_for(states_busy(c.R), s.max_q * group, c.R, sms);
    return c;
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

template <typename K>
cudaError_t allow_smem(K k, size_t bytes) {
    return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

template <typename T, int DP>
cudaError_t fwd_simple(const AttnShape& s, const AttnArgs& a, cudaStream_t st) {
    const size_t sm = (size_t(3) * kT * (DP + 4) + kT * kSP) * 4;
    cudaError_t e = allow_smem(attn_fwd_simple<T, DP>, sm);
    if (e != cudaSuccess) return e;
    attn_fwd_simple<T, DP><<<dim3(unsigned(row_tiles(s, kT)), unsigned(a.Hkv), unsigned(a.splits)), kThreads, sm, st>>>(a);
    return cudaGetLastError();
}

template <int DP, bool KV>
cudaError_t bwd_simple(const AttnArgs& a, int64_t tiles, cudaStream_t st) {
    const size_t sm = (size_t(4) * kT * (DP + 4) + 2 * kT * kSP) * 4;
    cudaError_t e = allow_smem(attn_bwd_simple<float, DP, KV>, sm);
    if (e != cudaSuccess) return e;
    attn_bwd_simple<float, DP, KV><<<dim3(unsigned(tiles), unsigned(a.Hkv), unsigned(a.splits)), kThreads, sm, st>>>(a);
    return cudaGetLastError();
}

template <typename F>
cudaError_t by_dim(int D, F f) {
    if (D <= 32) return f(std::integral_constant<int, 32>{});
    if (D <= 64) return f(std::integral_constant<int, 64>{});
    return f(std::integral_constant<int, 128>{});
}

}  // namespace

void attn_workspace(const AttnShape& s, int sms, size_t* fwd, size_t* bwd) {
    const Choice c = choose(s, sms);
    const size_t qh = size_t(s.n_q) * s.q_heads, kh = size_t(s.n_k) * s.kv_heads;
    const bool planes = c.engine == Engine::kPlanes;
    *fwd = c.fwd > 1 ? align256(c.fwd * qh * 4) + align256(c.fwd * qh * s.head_dim * 4) : 0;
    if (planes) *fwd += attn_planes_bytes(s, false);
    const size_t dq = c.dq > 1 ? c.dq * qh * s.head_dim * 4 : 0, dkv = c.dkv > 1 ? 2 * c.dkv * kh * s.head_dim * 4 : 0;
    *bwd = align256(qh * 4) + align256(std::max(dq, dkv));
    if (planes) *bwd += attn_planes_bytes(s, true);
}

AttnArgs attn_args(const AttnShape& s, const AttnTensors& t) {
    AttnArgs a = {};
    a.graphs = s.n_graphs;
    a.Hq = s.q_heads;
    a.Hkv = s.kv_heads;
    a.group = s.q_heads / s.kv_heads;
    a.D = s.head_dim;
    a.nq = s.n_q;
    a.nk = s.n_k;
    a.scale = float(s.scale);
    a.scale_log2 = float(s.scale * 1.4426950408889634);
    a.q_row = s.q_row, a.q_head = s.q_head, a.k_row = s.k_row, a.k_head = s.k_head;
    a.v_row = s.v_row, a.v_head = s.v_head, a.o_row = s.o_row, a.o_head = s.o_head;
    a.q_off = t.q_offsets, a.k_off = t.k_offsets, a.keep = t.keep;
    a.q = t.q, a.k = t.k, a.v = t.v, a.out = t.out, a.lse = t.lse;
    a.d_out = t.d_out, a.dq = t.dq, a.dk = t.dk, a.dv = t.dv;
    a.splits = 1;
    return a;
}

cudaError_t launch_attn_fwd(const AttnShape& s, const AttnTensors& t, void* ws, int sms, cudaStream_t st) {
    AttnArgs a = attn_args(s, t);
    const Choice c = choose(s, sms);
    a.splits = c.fwd;
    char* w = static_cast<char*>(ws);
    if (a.splits > 1) {
        const size_t n = size_t(a.splits) * a.nq * a.Hq;
        a.part_lse = reinterpret_cast<float*>(w);
        a.part_o = reinterpret_cast<float*>(w + align256(n * 4));
        w += align256(n * 4) + align256(n * a.D * 4);
    }
    cudaError_t e = cudaSuccess;
    switch (c.engine) {
        case Engine::kMma: e = launch_attn_fwd_mma(s.dtype, a, c.nt, c.fwd_tiles, st); break;
        case Engine::kPlanes:
            e = launch_attn_planes(a, w, sms, st);
            if (e == cudaSuccess) e = launch_attn_fwd_planes(a, w, c.fwd_tiles, st);
            break;
        case Engine::kCuda: e = by_dim(a.D, [&](auto d) { return fwd_simple<float, decltype(d)::value>(s, a, st); }); break;
    }
    if (e != cudaSuccess || a.splits == 1) return e;
    const unsigned blocks = unsigned((a.nq * a.Hq + 7) / 8);
    switch (s.dtype) {
        case UVU_F32: attn_fwd_join<float><<<blocks, kThreads, 0, st>>>(a); break;
        case UVU_BF16: attn_fwd_join<__nv_bfloat16><<<blocks, kThreads, 0, st>>>(a); break;
        default: attn_fwd_join<__half><<<blocks, kThreads, 0, st>>>(a); break;
    }
    return cudaGetLastError();
}

cudaError_t launch_attn_bwd(const AttnShape& s, const AttnTensors& t, void* ws, int sms, cudaStream_t st) {
    AttnArgs a = attn_args(s, t);
    a.delta = static_cast<float*>(ws);
    a.part_o = a.delta + align256(size_t(a.nq) * a.Hq * 4) / 4;
    const Choice c = choose(s, sms);
    const size_t dq = c.dq > 1 ? size_t(c.dq) * a.nq * a.Hq : 0, dkv = c.dkv > 1 ? 2 * size_t(c.dkv) * a.nk * a.Hkv : 0;
    void* planes = reinterpret_cast<char*>(a.part_o) + align256(std::max(dq, dkv) * a.D * 4);
    const auto with_type = [&](auto f) {
        switch (s.dtype) {
            case UVU_F32: f(float{}); break;
            case UVU_BF16: f(__nv_bfloat16{}); break;
            default: f(__half{}); break;
        }
        return cudaGetLastError();
    };
    const auto blocks = [](int64_t n) { return unsigned((n + kThreads - 1) / kThreads); };
    // dq, then dk and dv; the partial sums of one are joined before the other's are written
    const auto half = [&](bool kv) {
        a.splits = kv ? c.dkv : c.dq;
        const int64_t tiles = kv ? state_tiles(s, c.R) : row_tiles(s, c.R);
        cudaError_t e = cudaSuccess;
        switch (c.engine) {
            case Engine::kMma: e = launch_attn_bwd_mma(s.dtype, a, kv, tiles, st); break;
            case Engine::kPlanes: e = launch_attn_bwd_planes(a, planes, kv, tiles, st); break;
            case Engine::kCuda:
                e = by_dim(a.D, [&](auto d) {
                    constexpr int DP = decltype(d)::value;
                    return kv ? bwd_simple<DP, true>(a, tiles, st) : bwd_simple<DP, false>(a, tiles, st);
                });
                break;
        }
        if (e != cudaSuccess || a.splits == 1) return e;
        const int64_t n = kv ? a.nk * a.Hkv * a.D : a.nq * a.Hq * a.D;
        return with_type([&](auto t) {
            using T = decltype(t);
            attn_bwd_join<T><<<blocks(n), kThreads, 0, st>>>(n, a.splits, a.part_o, static_cast<T*>(kv ? a.dk : a.dq));
            if (kv) attn_bwd_join<T><<<blocks(n), kThreads, 0, st>>>(n, a.splits, a.part_o + a.splits * n, static_cast<T*>(a.dv));
        });
    };
    cudaError_t e = cudaSuccess;
    if (a.nq > 0)
        e = with_type([&](auto t) { attn_delta<decltype(t)><<<unsigned((a.nq * a.Hq + 7) / 8), kThreads, 0, st>>>(a); });
    if (e == cudaSuccess && c.engine == Engine::kPlanes) e = launch_attn_planes(a, planes, sms, st);
    if (e == cudaSuccess && a.dq && a.nq > 0) e = half(false);
    if (e == cudaSuccess && a.dk && a.nk > 0) e = half(true);
    return e;
}

// Status of the tensor-core attention kernels on the current device (bit 0: a bounded wait gave up).
cudaError_t attn_status(unsigned* word, bool reset) {
    unsigned a = 0, b = 0, c = 0;
    cudaError_t e = attn_fwd_mma_status(&a, reset);
    if (e == cudaSuccess) e = attn_bwd_mma_status(&b, reset);
    if (e == cudaSuccess) e = attn_planes_status(&c, reset);
    *word = a | b | c;
    return e;
}

}  // namespace uvu
