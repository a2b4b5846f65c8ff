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
// This file holds the launch choices and the kernels around the products: delta, and the joining of
// splits.  16-bit operands: attn_mma.cu, attn_mma_bwd.cu; fp32 operands: attn_planes.cu.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn.h"
#include "elem.h"

namespace uvu {
namespace {

constexpr int kThreads = 256;

// Joins the splits of a row: o = sum_s exp(lse_s - lse) o_s.  One warp per (row, head); lane s holds the
// weights of splits s and s + 32 (kMaxSplits = 64), the columns go by fours where D allows.
template <typename T>
__global__ void __launch_bounds__(kThreads) attn_fwd_join(AttnArgs a) {
    const int64_t rh = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int64_t total = a.nq * a.Hq;
    if (rh >= total) return;
    float x[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = lane + 32 * i < a.splits ? a.part_lse[(lane + 32 * i) * total + rh] : -INFINITY;
    float top = fmaxf(x[0], x[1]);
#pragma unroll
    for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
    float w[2], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w[i] = x[i] == -INFINITY ? 0.f : expf(x[i] - top);
        sum += w[i];
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    if (lane == 0) a.lse[rh] = sum == 0.f ? -INFINITY : top + logf(sum);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    T* po = static_cast<T*>(a.out) + (rh / a.Hq) * a.o_row + (rh % a.Hq) * a.o_head;
    const float* part = a.part_o + rh * a.D;
    const int64_t stride = total * a.D;
    auto weight = [&](int s) { return __shfl_sync(0xffffffffu, s < 32 ? w[0] : w[1], s & 31); };
    if (a.D % 4 == 0) {
        const int d = 4 * lane;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < a.splits; ++s) {
            const float ws = weight(s);
            if (d < a.D && ws != 0.f) {  // a piece without a kept state wrote zeros
                const float4 v = *reinterpret_cast<const float4*>(part + s * stride + d);
                o.x = fmaf(ws, v.x, o.x), o.y = fmaf(ws, v.y, o.y), o.z = fmaf(ws, v.z, o.z), o.w = fmaf(ws, v.w, o.w);
            }
        }
        if (d < a.D) {
            po[d] = narrow<T>(o.x * inv), po[d + 1] = narrow<T>(o.y * inv);
            po[d + 2] = narrow<T>(o.z * inv), po[d + 3] = narrow<T>(o.w * inv);
        }
    } else {
        for (int d0 = 0; d0 < a.D; d0 += 32) {
            float o = 0.f;
            for (int s = 0; s < a.splits; ++s) {
                const float ws = weight(s);
                if (d0 + lane < a.D && ws != 0.f) o = fmaf(ws, part[s * stride + d0 + lane], o);
            }
            if (d0 + lane < a.D) po[d0 + lane] = narrow<T>(o * inv);
        }
    }
}

// delta[row][head] = sum_d d_out out.  2^log2 lanes per (row, head), V columns at a time each.  For f16 also do2, in a
// second slice of the grid v2 (v's (state, kv head) in place of (row, head)), and the maxima are set to zero.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) attn_delta(AttnArgs a, int log2) {
    constexpr bool kNorms = __is_same(T, __half);
    const int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x, rh = i >> log2;
    const int lanes = 1 << log2, l = int(i) & (lanes - 1);
    const bool of_v = kNorms && blockIdx.y == 1;
    const int heads = of_v ? a.Hkv : a.Hq;
    const int64_t row = uint64_t(rh) < (1ull << 32) ? int64_t(uint32_t(rh) / uint32_t(heads)) : rh / heads;
    const bool on = row < (of_v ? a.nk : a.nq);
    float s = 0.f, square = 0.f;
    if (on && !(of_v && a.keep && !a.keep[row])) {
        const int64_t head = rh - row * heads, at = of_v ? row * a.v_row + head * a.v_head : row * a.o_row + head * a.o_head;
        for (int d = l * V; d < a.D; d += lanes * V) {
            const Vec<T, V> x = load_vec<T, V>(static_cast<const T*>(of_v ? a.v : a.d_out) + at + d);
            if (!of_v) {
                const Vec<T, V> y = load_vec<T, V>(static_cast<const T*>(a.out) + at + d);
#pragma unroll
                for (int k = 0; k < V; ++k) s = fmaf(widen(x.v[k]), widen(y.v[k]), s);
            }
            if constexpr (kNorms) {
#pragma unroll
                for (int k = 0; k < V; ++k) square = fmaf(widen(x.v[k]), widen(x.v[k]), square);
            }
        }
    }
    for (int k = lanes >> 1; k; k >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, k);
        if constexpr (kNorms) square += __shfl_xor_sync(0xffffffffu, square, k);
    }
    if (l == 0 && on) {
        if (!of_v) a.delta[rh] = s;
        if constexpr (kNorms) (of_v ? a.v2 : a.do2)[rh] = square;
    }
    if constexpr (kNorms) {
        unsigned* top = of_v ? a.v2_top : a.do2_top;
        for (int64_t t = i; t < int64_t(a.graphs) * a.Hkv; t += int64_t(gridDim.x) * kThreads) top[t] = 0;
    }
}

// do2_top and v2_top: a block takes the maximum of kTopRows packed rows (or states) of a graph and kv head.  The squares'
// bits are ordered like unsigned numbers (a NaN's above all), and a maximum does not depend on the order of the blocks.
constexpr int kTopRows = 2048;
__global__ void __launch_bounds__(kThreads) attn_tops(AttnArgs a) {
    __shared__ unsigned s_top;
    const bool of_v = blockIdx.z == 1;
    const int per = of_v ? 1 : a.group, h = blockIdx.y;
    if (int64_t(blockIdx.x) >= (of_v ? a.nk : a.nq) * per / kTopRows + a.graphs) return;
    if (threadIdx.x == 0) s_top = 0;
    const AttnTile tl = of_v ? attn_tile<kTopRows>(a.k_off, a.q_off, a.graphs, 1, blockIdx.x)
                             : attn_tile<kTopRows>(a.q_off, a.k_off, a.graphs, per, blockIdx.x);
    if (tl.graph < 0) return;
    const int n = int(min(int64_t(kTopRows), tl.rows - tl.row0));
    const float* x = of_v ? a.v2 : a.do2;
    unsigned top = 0;
#pragma unroll 4
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int64_t p = tl.row0 + i, r = per == 1 ? p : p / per;
        top = max(top, __float_as_uint(x[((tl.first + r) * a.Hkv + h) * per + (p - r * per)]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) atomicMax(&s_top, top);
    __syncthreads();
    if (threadIdx.x == 0) atomicMax((of_v ? a.v2_top : a.do2_top) + int64_t(tl.graph) * a.Hkv + h, s_top);
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

constexpr int kMaxSplits = 64;  // two weights per lane of the join

// Pieces of the inner axis where the tiles are fewer than the SMs: the fewest that leave at most a tenth of the last wave of
// `slots` blocks empty, within `waves` waves (or else the best of them), none shorter than four tiles.  The backward,
// whose pieces cost fp32 sums to join, takes one wave.  Single
// rows over 8 x 16384 states, 32/8 heads of 128: 101 us, 125 in the fewest pieces that give every SM one; 16 x 8192 states,
// 8/2 heads of 64, two blocks an SM: 25 and 29 us; one sequence unsplit 162 against 72 us (8 ragged ones to 16384 states).
int splits_for(int64_t tiles, int64_t inner, int R, int sms, int blocks_per_sm, int waves) {
    if (tiles <= 0 || tiles >= sms) return 1;
    const int64_t slots = int64_t(sms) * blocks_per_sm;
    const int64_t most = std::min({inner / (4 * R), waves * slots / tiles, int64_t(kMaxSplits)});
    int64_t best = 1;
    double filled = 0.;
    for (int64_t n = 1; n <= most && filled < .9; ++n) {
        const int64_t full = (n * tiles + slots - 1) / slots * slots;
        if (double(n * tiles) / double(full) > filled) best = n, filled = double(n * tiles) / double(full);
    }
    return int(best);
}

int64_t row_tiles(const AttnShape& s, int R) { return s.n_q * (s.q_heads / s.kv_heads) / R + s.n_graphs; }
int64_t state_tiles(const AttnShape& s, int R) { return s.n_k / R + s.n_graphs; }

struct Choice {
    bool planes;        // fp32 operands
    int nt;             // row tiles of 128 per block of the 16-bit forward
    int R;              // rows or states of a tile of the backward
    int64_t fwd_tiles;  // tile numbers of the forward
    int fwd, dq, dkv;   // splits
    bool hold, hold_q, hold_kv;  // walks of the forward, of dq, of dk and dv are long: their sums are held in memory
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
    c.planes = s.dtype == UVU_F32;
    c.R = c.planes ? plane_bwd_tile(s.head_dim) : 128;
    // Two row tiles a block once they fill the SMs (K and V loaded once for 256 rows, one tile's exponentials under the
    // other's products: 735 against 1207 us at 4 x 4096 rows, 8192 states, 16 heads of 128); below that one, which leaves no
    // SM idle (16 graphs of 256 rows and 300 states, 2 heads of 128: 11.9 against 15.2 us).
    c.nt = !c.planes && rows_busy(256) >= sms && s.max_q * group > 128 ? 2 : 1;
    c.fwd_tiles = row_tiles(s, 128 * c.nt);
    c.fwd = splits_for(rows_busy(128 * c.nt), s.max_k, 128, sms, c.nt == 1 && s.head_dim <= (c.planes ? 32 : 64) ? 2 : 1, 4);
    const auto held = [&](int64_t walk, int pieces) { return !c.planes && walk / pieces > 128 * attn_hold_tiles(s.dtype == UVU_F16); };
    c.hold = held(s.max_k, c.fwd);
    const int bwd_blocks = c.planes && s.head_dim <= 32 ? 2 : 1;
    c.dq = splits_for(rows_busy(c.R), s.max_k, 128, sms, bwd_blocks, 1);
    c.dkv = splits_for(states_busy(c.R), s.max_q * group, 128, sms, bwd_blocks, 1);
    c.hold_q = held(s.max_k, c.dq);
    c.hold_kv = held(s.max_q * group, c.dkv);
    return c;
}
bool joins_q(const Choice& c) { return c.dq > 1 || c.hold_q; }
bool joins_kv(const Choice& c) { return c.dkv > 1 || c.hold_kv; }

size_t tops_bytes(const AttnShape& s) { return size_t(2) * s.n_graphs * s.kv_heads * 4; }  // do2_top and v2_top

}  // namespace

void attn_workspace(const AttnShape& s, int sms, size_t* fwd, size_t* bwd) {
    const Choice c = choose(s, sms);
    const size_t qh = size_t(s.n_q) * s.q_heads, kh = size_t(s.n_k) * s.kv_heads;
    *fwd = c.fwd > 1 ? align256(c.fwd * qh * 4) + align256(c.fwd * qh * s.head_dim * 4) : 0;
    if (c.hold && c.fwd == 1) *fwd = align256(qh * s.head_dim * 4);
    if (c.planes) *fwd += attn_planes_bytes(s, false);
    const size_t dq = joins_q(c) ? c.dq * qh * s.head_dim * 4 : 0, dkv = joins_kv(c) ? 2 * c.dkv * kh * s.head_dim * 4 : 0;
    *bwd = align256(qh * 4) + align256(dq) + align256(dkv);
    if (s.dtype == UVU_F16) *bwd += align256(qh * 4) + align256(kh * 4) + align256(tops_bytes(s));
    if (c.planes) *bwd += attn_planes_bytes(s, true);
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
    a.hold = c.hold;
    if (c.hold && c.fwd == 1) a.part_o = reinterpret_cast<float*>(w);
    cudaError_t e = cudaSuccess;
    if (c.planes) {
        e = launch_attn_planes(a, w, sms, st);
        if (e == cudaSuccess) e = launch_attn_fwd_planes(a, w, c.fwd_tiles, st);
    } else {
        e = launch_attn_fwd_mma(s.dtype, a, c.nt, c.fwd_tiles, st);
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
    const Choice c = choose(s, sms);
    const bool want_q = a.dq && a.nq > 0, want_kv = a.dk && a.nk > 0;
    const int64_t n_q = a.nq * a.Hq * a.D, n_kv = a.nk * a.Hkv * a.D;
    char* w = static_cast<char*>(ws);
    const auto take = [&](size_t bytes) {
        char* p = w;
        w += align256(bytes);
        return reinterpret_cast<float*>(p);
    };
    a.delta = take(size_t(a.nq) * a.Hq * 4);
    a.splits_q = c.dq, a.splits_kv = c.dkv;
    a.part_q = joins_q(c) ? take(size_t(c.dq) * n_q * 4) : nullptr;
    a.part_kv = joins_kv(c) ? take(2 * size_t(c.dkv) * n_kv * 4) : nullptr;
    a.hold = c.hold_q || c.hold_kv;
    a.kv_tiles = want_kv ? state_tiles(s, c.R) : 0;
    a.q_tiles = want_q ? row_tiles(s, c.R) : 0;
    if (s.dtype == UVU_F16) {
        a.do2 = take(size_t(a.nq) * a.Hq * 4);
        a.v2 = take(size_t(a.nk) * a.Hkv * 4);
        a.do2_top = reinterpret_cast<unsigned*>(take(tops_bytes(s)));
        a.v2_top = a.do2_top + size_t(a.graphs) * a.Hkv;
    }
    a.q_first = s.max_k > s.max_q * a.group;
    if ((a.kv_tiles + a.q_tiles) * a.Hkv > INT32_MAX) return cudaErrorInvalidConfiguration;
    const auto with_type = [&](auto f) {
        switch (s.dtype) {
            case UVU_F32: f(float{}); break;
            case UVU_BF16: f(__nv_bfloat16{}); break;
            default: f(__half{}); break;
        }
        return cudaGetLastError();
    };
    const auto blocks = [](int64_t n) { return unsigned((n + kThreads - 1) / kThreads); };
    cudaError_t e = cudaSuccess;
    if (c.planes) {
        e = launch_attn_planes(a, w, sms, st);
        if (e == cudaSuccess) e = launch_attn_bwd_planes(a, w, st);
    } else {
        if (a.nq > 0)  // without a row nothing needs delta or a scale
            e = with_type([&](auto t) {
                using T = decltype(t);
                constexpr int V = 16 / int(sizeof(T));
                constexpr bool kNorms = __is_same(T, __half);
                const uintptr_t any = reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.d_out) |
                                      uintptr_t(a.o_row | a.o_head) * sizeof(T) |
                                      (kNorms ? reinterpret_cast<uintptr_t>(a.v) | uintptr_t(a.v_row | a.v_head) * sizeof(T) : 0);
                const bool vec = a.D % V == 0 && (any & 15u) == 0;
                int log2 = 0;
                while (log2 < 5 && (1 << log2) * (vec ? V : 1) < a.D) ++log2;
                const dim3 n(blocks((kNorms ? std::max(a.nq * a.Hq, a.nk * a.Hkv) : a.nq * a.Hq) << log2), kNorms ? 2 : 1);
                vec ? attn_delta<T, V><<<n, kThreads, 0, st>>>(a, log2) : attn_delta<T, 1><<<n, kThreads, 0, st>>>(a, log2);
                if (kNorms)
                    attn_tops<<<dim3(unsigned(std::max(a.nq * a.group, a.nk) / kTopRows + a.graphs), unsigned(a.Hkv), 2), kThreads, 0,
                                st>>>(a);
            });
        if (e == cudaSuccess) e = launch_attn_bwd_mma(s.dtype, a, st);
    }
    if (e != cudaSuccess) return e;
    return with_type([&](auto t) {
        using T = decltype(t);
        const auto join = [&](int64_t n, int splits, const float* part, void* dst) {
            attn_bwd_join<T><<<blocks(n), kThreads, 0, st>>>(n, splits, part, static_cast<T*>(dst));
        };
        if (want_q && joins_q(c)) join(n_q, c.dq, a.part_q, a.dq);
        if (want_kv && joins_kv(c)) {
            join(n_kv, c.dkv, a.part_kv, a.dk);
            join(n_kv, c.dkv, a.part_kv + c.dkv * n_kv, a.dv);
        }
    });
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
