// Attention of fp32 operands on the 16-bit tensor cores, with fp32 accuracy.
//
// An fp32 value is the exact sum of three bf16 values, its leading 8 significant bits, the next 8 and
// the last 8 (x = x0 + x1 + x2, each remainder cut to its upper half: bf16 has the exponent range of
// fp32, and a cut of 8 bits leaves an exact remainder).  A product keeps the terms x_i y_j with
// i + j <= 2; what is dropped is 2^-24 of it.  That is six bf16 products, at 1/6 of their rate still several
// times the CUDA cores' fp32 rate.
//   - A first kernel writes the planes of q, k, v (and d_out) to the workspace, [row][head][3][PS] with
//     PS = 16, 32, 64 or 128 columns a plane (zeros past head_dim), so that the loaders below move them like any 16-bit
//     operand.  Infinities and NaN stay in x0.
//   - S (and dP): the six products are issued smallest first into one accumulator.
//   - P (and dS) are cut into planes by the threads that form them; with X = [X0 | X1 | X2] side by side in
//     the tile, P0 X, P1 [X0 | X1] and P2 X0 land in columns by order of magnitude: the sums of the small terms
//     are apart from the large ones, and the threads add them.
//   - Tensor memory sums each tile afresh; the sums over tiles are fp32 registers (each accumulating
//     instruction cuts a sum in tensor memory by up to 2^-23 of it, and 3000 rows showed it).  Where the backward has no
//     registers for that, tensor memory sums 512 rows, the small terms in columns of their own (or 64 rows, all in the
//     same), and the threads add that to the gradient in memory.
// Masks, splits and bounded waits as in the 16-bit kernels.
// Measured, forward and backward at 4 x 2048 rows and 4096 states, in TFLOP/s of the formula's products: 142 (4 heads of 64),
// 103 (4 of 32), 67 (8 of 16), 70 (4 of 128); forward alone at 64 153.  Six products for one: the tensor cores' rate over
// six would be 309.  Bound by the waits between the roles, and at small head dimensions by the least time of an
// instruction, about 40 clocks however few its columns.
#include "attn_mma.h"

namespace uvu {
namespace {

// ----------------------------------------------------------------------------------- planes

struct PlaneJob {
    const float* x;
    int64_t row, head;  // strides
    int64_t rows;
    int heads;
    uint16_t* out;  // [rows][heads][3][PS]
    bool vec;       // fours of columns are 16-byte aligned
};
struct PlaneJobs {
    PlaneJob j[4];
    int D;
    bool vec_o;  // of out and d_out
};

// The planes of two values, packed: the leading plane in p[0].
__device__ __forceinline__ void cut2(float x, float y, uint32_t (&p)[3]) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    p[0] = __byte_perm(a, b, 0x7632);
    const float x1 = x - __uint_as_float(a & 0xffff0000u), y1 = y - __uint_as_float(b & 0xffff0000u);
    const uint32_t c = __float_as_uint(x1), d = __float_as_uint(y1);
    p[1] = __byte_perm(c, d, 0x7632);
    p[2] = __byte_perm(__float_as_uint(x1 - __uint_as_float(c & 0xffff0000u)), __float_as_uint(y1 - __uint_as_float(d & 0xffff0000u)), 0x7632);
}

// A thread per 8 columns of a (row, head), 64 rows a block; the backward's last slice of the grid forms delta, a
// thread per (row, head).
template <int PS>
__global__ void __launch_bounds__(256) attn_planes(PlaneJobs jobs, AttnArgs a) {
    constexpr int kChunks = PS / 8, kBlockRows = 64;
    if (blockIdx.y == 4) {
        for (int64_t r0 = int64_t(blockIdx.x) * kBlockRows; r0 < a.nq; r0 += int64_t(gridDim.x) * kBlockRows) {
            const int n = int(min(int64_t(kBlockRows), a.nq - r0)) * a.Hq;
            for (int i = threadIdx.x; i < n; i += 256) {
                const int r = i / a.Hq, h = i - r * a.Hq;
                const int64_t at = (r0 + r) * a.o_row + h * a.o_head;
                const float *x = static_cast<const float*>(a.d_out) + at, *y = static_cast<const float*>(a.out) + at;
                float s = 0.f;
                if (jobs.vec_o) {
                    for (int d = 0; d < a.D; d += 4) {
                        const float4 u = *reinterpret_cast<const float4*>(x + d), v = *reinterpret_cast<const float4*>(y + d);
                        s = fmaf(u.x, v.x, fmaf(u.y, v.y, fmaf(u.z, v.z, fmaf(u.w, v.w, s))));
                    }
                } else {
                    for (int d = 0; d < a.D; ++d) s = fmaf(x[d], y[d], s);
                }
                a.delta[(r0 + r) * a.Hq + h] = s;
            }
        }
        return;
    }
    const PlaneJob& j = jobs.j[blockIdx.y];
    const int per = j.heads * kChunks;
    for (int64_t r0 = int64_t(blockIdx.x) * kBlockRows; r0 < j.rows; r0 += int64_t(gridDim.x) * kBlockRows) {
        const int n = int(min(int64_t(kBlockRows), j.rows - r0)) * per;
        for (int i = threadIdx.x; i < n; i += 256) {
            const int rr = i / per, e = i - rr * per;
            const int64_t r = r0 + rr;
            const int h = e / kChunks, c = e % kChunks * 8;
            const float* x = j.x + r * j.row + h * j.head + c;
            float v[8];
            if (j.vec) {
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const float4 q = c + k < jobs.D ? *reinterpret_cast<const float4*>(x + k) : make_float4(0.f, 0.f, 0.f, 0.f);
                    v[k] = q.x, v[k + 1] = q.y, v[k + 2] = q.z, v[k + 3] = q.w;
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = c + k < jobs.D ? x[k] : 0.f;
            }
            uint32_t w[3][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t p[3];
                cut2(v[2 * k], v[2 * k + 1], p);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float z = v[2 * k + i];
                    if (!isfinite(z)) {  // whole in the leading plane (a NaN's upper bits alone could read as infinity)
                        const uint32_t half = isnan(z) ? 0x7fffu : __float_as_uint(z) >> 16, keep = i ? 0x0000ffffu : 0xffff0000u;
                        p[0] = (p[0] & keep) | (half << (16 * i));
                        p[1] &= keep;
                        p[2] &= keep;
                    }
                }
#pragma unroll
                for (int q = 0; q < 3; ++q) w[q][k] = p[q];
            }
            uint16_t* o = j.out + (r * j.heads + h) * (3 * PS) + c;
#pragma unroll
            for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4*>(o + q * PS) = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
        }
    }
}

// An operand's planes in the workspace.
struct Planes {
    const uint16_t *q, *k, *v, *d_out;
};

template <int PS>
constexpr int kPanels = (3 * PS + 63) / 64;

// A tile of plane rows, all panels of a row together: the thread's rows are `step` bytes apart from p on (its chunk
// included); those that use(i) refuses are zeros.  ALL: every row is used.
template <int PS, int ROWS, bool ALL, typename Use>
__device__ __forceinline__ void load_plane_rows(uint32_t dst, const char* p, int64_t step, int t, Use use) {
    constexpr int kLast = (3 * PS - 64 * (kPanels<PS> - 1)) / 8;  // chunks of the last panel
    const uint32_t to = dst + tile_offset(t >> 3, t & 7);
    const bool last = (t & 7) < kLast;
#pragma unroll 4
    for (int i = 0; i < ROWS / 8; ++i) {
        const uint32_t bytes = ALL || use(i) ? 16 : 0;
#pragma unroll
        for (int k = 0; k < kPanels<PS>; ++k)
            if (k + 1 < kPanels<PS> || last) copy16(to + uint32_t(i * 1024 + k * ROWS * 128), p + k * 128, bytes);
        p += step;
    }
}
static_assert(kLoadThreads == 64, "eight rows of eight chunks a step");
template <int PS, int ROWS>
__device__ __forceinline__ void load_planes(uint32_t dst, const char* src, int64_t stride, int t, const StateMask<ROWS>& mask) {
    const char* p = src + (t >> 3) * stride + (t & 7) * 16;
    if (mask.all()) {
        load_plane_rows<PS, ROWS, true>(dst, p, 8 * stride, t, [](int) { return true; });
    } else {
        const uint32_t mine = mask.template every<8>(t >> 3);
        load_plane_rows<PS, ROWS, false>(dst, p, 8 * stride, t, [&](int i) { return (mine >> i) & 1; });
    }
}
// Packed rows, as load_packed().
template <int PS, int ROWS, bool ZERO>
__device__ __forceinline__ void load_planes_packed(uint32_t dst, const char* base, int64_t row, int64_t head, int group, int64_t r0,
                                                   int rows, int t) {
    if (group == 1 && (ZERO || rows >= ROWS)) {
        const char* p = base + (r0 + (t >> 3)) * row + (t & 7) * 16;
        if (rows >= ROWS)
            load_plane_rows<PS, ROWS, true>(dst, p, 8 * row, t, [](int) { return true; });
        else
            load_plane_rows<PS, ROWS, false>(dst, p, 8 * row, t, [&](int i) { return (t >> 3) + 8 * i < rows; });
        return;
    }
#pragma unroll
    for (int p = 0; p < kPanels<PS>; ++p) {
        const LoadMap<3, ROWS> m(t, 3 * PS - 64 * p < 64 ? 3 * PS - 64 * p : 64);
        load_packed<true, ZERO>(dst + p * ROWS * 128, base + p * 128, row, head, group, r0, rows, m);
    }
}

// The six products of S (or dP) = A B^T, smallest first; panels of `rows` x 128 bytes.
template <int PS>
__device__ __forceinline__ void six_products(uint32_t lead, uint32_t d, uint32_t a, int a_panel, uint32_t b, int b_panel, uint32_t id) {
    constexpr int kStep = PS / 16;
    constexpr int kPair[6][2] = {{2, 0}, {1, 1}, {0, 2}, {1, 0}, {0, 1}, {0, 0}};
    bool add = false;
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
        for (int s = 0; s < kStep; ++s) {
            mma_ss(lead, d, desc_cols(a, kPair[i][0] * kStep + s, a_panel), desc_cols(b, kPair[i][1] * kStep + s, b_panel), id, add);
            add = true;
        }
}

// N (32 or 16) values of a row to the three planes of a 16-bit operand in tensor memory.
template <int N>
__device__ __forceinline__ void store_planes(const float (&x)[N], uint32_t hi, uint32_t mid, uint32_t lo) {
    uint32_t w[3][N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        uint32_t p[3];
        cut2(x[2 * i], x[2 * i + 1], p);
#pragma unroll
        for (int q = 0; q < 3; ++q) w[q][i] = p[q];
    }
    const uint32_t at[3] = {hi, mid, lo};
#pragma unroll
    for (int q = 0; q < 3; ++q) {
        if constexpr (N == 32)
            tmem_st16(at[q], w[q]);
        else
            tmem_st8(at[q], w[q]);
    }
}
__device__ __forceinline__ void load_columns(uint32_t a, float (&v)[32]) { tmem_ld32(a, v); }
__device__ __forceinline__ void load_columns(uint32_t a, float (&v)[16]) { tmem_ld16(a, v); }
__device__ __forceinline__ void load_columns(uint32_t a, float (&v)[8]) { tmem_ld8(a, v); }

// Column of 16-row block s of a plane-0 operand that its two warpgroups wrote over their halves (`half`
// columns each) of the fp32 tile.
__device__ __forceinline__ uint32_t block_column(int s, int half) {
    return uint32_t(s / (half / 16) * half + s % (half / 16) * 8);
}

// acc[i] += the sum of column i of N in each of ORDERS blocks of PS columns from `a` on, the small terms (the last block) first:
// added to acc one by one they would be lost in a long walk's sum (out over 2^20 states of one sign: off by 2.1e-5, so by 1.7e-6).
template <int N, int PS, int ORDERS>
__device__ __forceinline__ void add_columns(uint32_t a, float* acc) {
    constexpr int kBlock = N < 16 ? N : 16;
#pragma unroll
    for (int b = 0; b < N / kBlock; ++b) {
        float v[ORDERS][kBlock];
#pragma unroll
        for (int o = 0; o < ORDERS; ++o) load_columns(a + o * PS + kBlock * b, v[o]);
#pragma unroll
        for (int o = 0; o < ORDERS; ++o) tmem_wait_ld(v[o]);
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
            float sum = v[ORDERS - 1][i];
#pragma unroll
            for (int o = ORDERS - 2; o >= 0; --o) sum += v[o][i];
            acc[kBlock * b + i] += sum;
        }
    }
}

// N columns from c0 on of a row of D fp32 values, times scale; `add`: to what this thread stored there before (as
// reductions, which it does not wait for; one thread to an element, so their order is its own).
template <int N>
__device__ __forceinline__ void store_row(float* dst, const float* v, float scale, int c0, int D, bool add = false) {
    const bool vec = D % 4 == 0 && (reinterpret_cast<uintptr_t>(dst) & 15u) == 0;
    if (add) {
        if (vec) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                if (c0 + i < D)
                    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(dst + c0 + i), "f"(v[i] * scale),
                                 "f"(v[i + 1] * scale), "f"(v[i + 2] * scale), "f"(v[i + 3] * scale)
                                 : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (c0 + i < D) atomicAdd(dst + c0 + i, v[i] * scale);
        }
    } else if (vec) {
#pragma unroll
        for (int i = 0; i < N; i += 4)
            if (c0 + i < D)
                *reinterpret_cast<float4*>(dst + c0 + i) = make_float4(v[i] * scale, v[i + 1] * scale, v[i + 2] * scale, v[i + 3] * scale);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (c0 + i < D) dst[c0 + i] = v[i] * scale;
    }
}

// ----------------------------------------------------------------------------------- forward

// PS <= 32: one warpgroup per row tile, state tiles of 64, 256 columns of tensor memory and at most 102 KB: two CTAs an
// SM, whose products and exponentials overlap.  Above, one CTA an SM whose two warpgroups share a tile, warpgroup w taking
// the w-th half of a row's columns; state tiles of 128, or of 64 where a tile's planes would not fit beside Q's (PS = 128).
template <int PS>
struct FwdPlan {
    static constexpr int kGroups = PS <= 32 ? 1 : 2, kWarps = 4 * kGroups, kThreads = (kWarps + 1 + kLoadWarps) * 32;
    static constexpr int kState = PS == 64 ? 128 : 64, kHalfState = kState / kGroups, kPanel = kState * 128;
    static constexpr int kTile = kPanels<PS> * kPanelBytes, kStep = kPanels<PS> * kPanel;
    static constexpr int kStages = PS == 128 ? 2 : PS == 64 ? 3 : PS == 32 ? 4 : 8;
    static constexpr int kRing = kTile, kMasks = kRing + kStages * kStep, kMax = kMasks + 8 * kState * 4, kBars = kMax + 2 * 2 * kRows * 4;
    static constexpr int kTotal = kBars + 512 + 1024;  // barriers, alignment slack
    // tensor memory: S (plane 0 of P written over it), planes 1 and 2 of P, O by order
    static constexpr uint32_t kMid = kState, kLo = kState + kState / 2, kO = 2 * kState, kColumns = kO + 3 * PS <= 256 ? 256 : 512;
};

template <int PS>
__global__ void __launch_bounds__(FwdPlan<PS>::kThreads, FwdPlan<PS>::kColumns == 256 ? 2 : 1) attn_fwd_planes(AttnArgs a, Planes x) {
    using F = FwdPlan<PS>;
    constexpr int kHalf = PS / F::kGroups, kRing = 8, kBlocks = F::kHalfState / 32;  // 32-column blocks of a warpgroup
    extern __shared__ unsigned char smem_raw[];
    __shared__ int s_dead, s_kept;  // s_kept: a mask has kept one of the piece's states
    __shared__ uint32_t s_tmem;
    const AttnTile tl = attn_tile<kRows>(a.q_off, a.k_off, a.graphs, a.group, blockIdx.x);
    if (tl.graph < 0) return;
    const int h = blockIdx.y, split = blockIdx.z;
    const int64_t q0 = tl.first, k0 = tl.other;
    const Piece kr = piece_of(tl.n, split, a.splits);
    const int n_tiles = uniform(int((kr.hi - kr.lo + F::kState - 1) / F::kState));
    const int n_rows = uniform(int(min(tl.rows - tl.row0, int64_t(kRows))));
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = uniform(smem_u32(smem));
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t q_full = sb + F::kBars, s_full = q_full + 8, p_full = s_full + 8, o_full = p_full + 8, fin = o_full + 8,
                   pair = fin + 8, full = pair + 32, empty = full + 8 * F::kStages, m_full = empty + 8 * F::kStages;
    if (threadIdx.x == 0) {
        s_dead = s_kept = 0;
        bar_init(q_full, kLoadThreads);
        bar_init(s_full, 1);
        bar_init(p_full, F::kWarps);
        bar_init(o_full, 1);
        bar_init(fin, 1);
        for (int i = 0; i < 4; ++i) bar_init(pair + 8 * i, 2);
        for (int s = 0; s < F::kStages; ++s) {
            bar_init(full + 8 * s, kLoadThreads);
            bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < kRing; ++s) bar_init(m_full + 8 * s, kLoadThreads);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == F::kWarps) tmem_alloc(smem_u32(&s_tmem), F::kColumns);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(&s_tmem));
    volatile int* dead = &s_dead;
    unsigned* status = &attn_status_word;
    float* biases = reinterpret_cast<float*>(smem + F::kMasks);
    // the bias of tile j: every tile's with a mask, else the last one's where it is not full
    const bool tail = (kr.hi - kr.lo) % F::kState != 0;
    auto masked = [&](int j) { return a.keep || (tail && j == n_tiles - 1); };
    auto slot = [&](int j) { return a.keep ? j % kRing : 0; };

    if (warp < F::kWarps) {
        // ------------------------------------------------------------------------ softmax
        const int w = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const bool work = quad * 32 < n_rows;
        const uint32_t lanes = uint32_t(quad * 32) << 16, base_t = tmem + lanes;
        const float c = a.scale_log2;
        float* s_max = reinterpret_cast<float*>(smem + F::kMax);  // [turn][warpgroup][row]
        float m = -INFINITY, l = 0.f, acc[kHalf];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) acc[i] = 0.f;
        int turn = 0;
        bool ok = true;
        // the partner warpgroup's value of the same row
        auto exchange = [&](float v, float& other) {
            if constexpr (F::kGroups == 1) return true;
            float* s = s_max + (turn & 1) * 2 * kRows;
            s[w * kRows + row] = v;
            __syncwarp();
            if (lane == 0) bar_arrive(pair + 8 * quad);
            if (!warp_wait(pair + 8 * quad, turn & 1, dead, status)) return false;
            other = s[(1 - w) * kRows + row];
            ++turn;
            return true;
        };
        // this warpgroup's half of the columns of O, all orders
        auto add_o = [&]() { add_columns<kHalf, PS, 3>(base_t + F::kO + w * kHalf, acc); };
        for (int j = 0; j < n_tiles; ++j) {
            const bool biased = masked(j);
            const float* bias = biases + slot(j) * F::kState + F::kHalfState * w;
            if (biased) {
                ok = warp_wait(m_full + 8 * slot(j), a.keep ? (j / kRing) & 1 : 0, dead, status);
                if (!ok) break;
            }
            ok = warp_wait(s_full, j & 1, dead, status);
            if (!ok) break;
            fence_after();
            if (work) {
                if (j > 0) add_o();  // O of the tile before is complete when S of this one is
                float v[kBlocks][32];
                float top = -INFINITY;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) tmem_ld32(base_t + F::kHalfState * w + 32 * b, v[b]);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    tmem_wait_ld(v[b]);
                    if (biased) add_bias(v[b], bias + 32 * b);
                    top = fmaxf(top, row_max(v[b]));
                }
                float other = -INFINITY;
                ok = exchange(top, other);
                if (!ok) break;
                const float mn = fmaxf(m, fmaxf(top, other) * c), base = mn == -INFINITY ? 0.f : mn;
                const float f = exp2_approx(m - base);
                m = mn;
                l *= f;
#pragma unroll
                for (int i = 0; i < kHalf; ++i) acc[i] *= f;
                F2 sum[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    exp_row(v[b], F2(c, c), F2(-base, -base), sum);
                    store_planes(v[b], base_t + F::kHalfState * w + 16 * b, base_t + F::kMid + F::kHalfState / 2 * w + 16 * b,
                                 base_t + F::kLo + F::kHalfState / 2 * w + 16 * b);
                }
                const float2 s2 = (sum[0] + sum[1]).both();
                l += s2.x + s2.y;
                tmem_wait_st();
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_full);
        }
        if (ok && n_tiles > 0) {
            ok = warp_wait(o_full, 0, dead, status);
            fence_after();
        }
        if (ok && work) {
            if (n_tiles > 0) add_o();
            float other = 0.f;
            if (exchange(l, other)) {
                // nothing to attend to, whatever q holds: 0
                const float sum = a.keep && !*static_cast<volatile int*>(&s_kept) ? 0.f : w ? other + l : l + other;
                const int64_t p = tl.row0 + row;
                const int64_t r = q0 + p / a.group, head = int64_t(h) * a.group + p % a.group;
                const int64_t rh = (int64_t(split) * a.nq + r) * a.Hq + head;
                if (row < n_rows) {
                    if (w == 0)
                        (a.splits > 1 ? a.part_lse[rh] : a.lse[r * a.Hq + head]) = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
                    if (sum == 0.f) {
#pragma unroll
                        for (int i = 0; i < kHalf; ++i) acc[i] = 0.f;
                    }
                    float* dst = a.splits > 1 ? a.part_o + rh * a.D : static_cast<float*>(a.out) + r * a.o_row + head * a.o_head;
                    store_row<kHalf>(dst, acc, sum == 0.f ? 0.f : 1.f / sum, w * kHalf, a.D);
                }
            }
        }
    } else if (warp == F::kWarps) {
        // ----------------------------------------------------------------- matrix instructions
        {
            const uint32_t lead = elect_lane();
            constexpr uint32_t o = F::kO;
            const uint32_t id_s = mma_desc<__nv_bfloat16>(F::kState, false), id3 = mma_desc<__nv_bfloat16>(3 * PS <= 256 ? 3 * PS : 256, true),
                           id2 = mma_desc<__nv_bfloat16>(2 * PS, true), id1 = mma_desc<__nv_bfloat16>(PS, true);
            auto stage = [&](int i) { return sb + uint32_t(F::kRing + (i % F::kStages) * F::kStep); };
            auto wait_stage = [&](int i) {
                if (!warp_wait(full + 8 * (i % F::kStages), (i / F::kStages) & 1, dead, status)) return false;
                fence_async();
                return true;
            };
            auto scores = [&](int j) {
                six_products<PS>(lead, tmem, sb, kPanelBytes, stage(2 * j), F::kPanel, id_s);
                mma_commit(lead, s_full);
                mma_commit(lead, empty + 8 * ((2 * j) % F::kStages));
            };
            bool ok = n_tiles > 0 && warp_wait(q_full, 0, dead, status) && wait_stage(0);
            if (ok) scores(0);
            for (int j = 0; j < n_tiles && ok; ++j) {
                ok = wait_stage(2 * j + 1) && warp_wait(p_full, j & 1, dead, status);
                if (!ok) break;
                fence_after();
                const uint32_t v = stage(2 * j + 1);
#pragma unroll
                for (int s = 0; s < F::kState / 16; ++s) {
                    const uint32_t hi = tmem + block_column(s, F::kHalfState), mid = tmem + F::kMid + 8 * s, lo = tmem + F::kLo + 8 * s;
                    const uint64_t v0 = desc_rows(v, s, F::kPanel);
                    if constexpr (3 * PS <= 256) {
                        mma_ts(lead, tmem + o, hi, v0, id3, s > 0);
                    } else {  // 256 columns at most
                        mma_ts(lead, tmem + o, hi, v0, id2, s > 0);
                        mma_ts(lead, tmem + o + 2 * PS, hi, desc_rows(v, s, F::kPanel, 2 * PS), id1, s > 0);
                    }
                    mma_ts(lead, tmem + o + PS, mid, v0, id2, true);
                    mma_ts(lead, tmem + o + 2 * PS, lo, v0, id1, true);
                }
                mma_commit(lead, empty + 8 * ((2 * j + 1) % F::kStages));
                if (j + 1 < n_tiles) {
                    ok = wait_stage(2 * j + 2);
                    if (ok) scores(j + 1);
                } else {
                    mma_commit(lead, o_full);
                }
            }
            mma_commit(lead, fin);
            bar_wait_last(fin, 0, status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------------- loaders
        const int t = threadIdx.x - (F::kWarps + 1) * 32;
        if (n_tiles > 0) {
            constexpr int64_t kHead = 3 * PS * 2;  // bytes of a (row, head)
            load_planes_packed<PS, kRows, false>(sb, reinterpret_cast<const char*>(x.q) + (q0 * a.Hq + int64_t(h) * a.group) * kHead,
                                          a.Hq * kHead, kHead, a.group, tl.row0, n_rows, t);
            copy_arrive(q_full);
            const char* K = reinterpret_cast<const char*>(x.k) + ((k0 + kr.lo) * a.Hkv + h) * kHead;
            const char* V = reinterpret_cast<const char*>(x.v) + ((k0 + kr.lo) * a.Hkv + h) * kHead;
            const int64_t stride = a.Hkv * kHead;
            StateMask<F::kState> mask(a.keep ? a.keep + k0 : nullptr, kr.lo, kr.hi);
            auto load = [&](int i, const char* src) {
                if (i >= F::kStages && !warp_wait(empty + 8 * (i % F::kStages), (i / F::kStages - 1) & 1, dead, status))
                    return false;
                const uint32_t dst = sb + uint32_t(F::kRing + (i % F::kStages) * F::kStep);
                load_planes<PS>(dst, src, stride, t, mask);
                copy_arrive(full + 8 * (i % F::kStages));
                return true;
            };
            for (int j = 0; j < n_tiles; ++j) {
                mask.next();
                if (!load(2 * j, K)) break;
                if (masked(j)) {
                    if (t == 0 && mask.any()) s_kept = 1;
                    write_bias(biases + slot(j) * F::kState, mask, t);
                    bar_arrive(m_full + 8 * slot(j));
                }
                if (!load(2 * j + 1, V)) break;
                K += F::kState * stride;
                V += F::kState * stride;
            }
            copy_wait_all();
        }
    }
    fence_before();
    __syncthreads();
    if (warp == F::kWarps) {
        fence_after();
        tmem_free(tmem, F::kColumns);
    }
}

// ---------------------------------------------------------------------------------- backward

// The walk, its order and the roles as in the 16-bit backward, in steps of 32 or 64 walked rows.  Tensor memory:
// S with plane 0 of P over it, planes 1 and 2 of P, dP and the planes of dS likewise, then the sums.
//   PS <= 32   one warpgroup, steps of 32, 256 columns of tensor memory and at most 98 KB: two CTAs an SM.  The sums
//              of 512 rows in tensor memory.
//   PS = 64    two warpgroups, steps of 64 (the planes of two resident tiles leave room for four such stages).  The
//              sums of one step in tensor memory, the others in registers.
//   PS = 128   two warpgroups, steps of 32, resident tiles of 64 rows (the instructions still take 128: the upper half
//              reads whatever follows in shared memory, into lanes that nobody reads).  The sums of 512 rows in tensor memory
//              for dq; of 64 rows for dk and dv, whose small terms go to the columns of the leading ones, as tensor
//              memory has no others (69 TFLOP/s forward and backward at 4 x 2048 rows, 4096 states, 4 heads; with dk and dv in
//              two halves of 64 columns, which forms S and dP twice, 46).
// A gradient's leading terms are in PS columns, its small ones in PS more.
template <int PS, bool KV>
struct BwdPlan {
    static constexpr bool kHeld = PS != 64;  // sums of kFlush steps in tensor memory, else of one
    static constexpr int kGroups = PS <= 32 ? 1 : 2, kWarps = 4 * kGroups;
    static constexpr int kOwn = PS == 128 ? 64 : 128, kWalk = PS == 64 ? 64 : 32, kHalf = kWalk / kGroups;
    static constexpr int kOwnPanel = kOwn * 128, kPanel = kWalk * 128;
    static constexpr int kTile = kPanels<PS> * kOwnPanel, kStep = kPanels<PS> * kPanel, kStages = PS == 16 ? 8 : 4;
    static constexpr int kHalfRing = kStages / 2, kRing = 2 * kTile, kAux = kRing + kStages * kStep;
    static constexpr int kAuxBytes = (KV ? 2 : 1) * kWalk * 4;  // -lse and -delta of the step, or the states' bias
    static constexpr int kBars = kAux + kHalfRing * kAuxBytes, kTotal = kBars + 512 + 1024;
    static constexpr uint32_t kP1 = kWalk, kP2 = kP1 + kWalk / 2, kDp = 2 * kWalk, kD1 = kDp + kWalk, kD2 = kD1 + kWalk / 2, kG = 4 * kWalk;
    static constexpr bool kTogether = PS == 128 && KV;
    static constexpr int kFlush = (kTogether ? 64 : 512) / kWalk, kGrad = kTogether ? PS : 2 * PS;  // steps, columns of a gradient's sums
    static constexpr uint32_t kColumns = kG + 2 * kGrad <= 256 ? 256 : 512;
};

template <int PS, bool KV>
__device__ __forceinline__ void bwd_tile(const AttnArgs& a, const Planes& x, int64_t tile, int h) {
    using B = BwdPlan<PS, KV>;
    constexpr int kCols = KV ? PS : PS / B::kGroups;  // columns of a gradient that a thread writes
    constexpr float kLog2e = 1.4426950408889634f;
    extern __shared__ unsigned char smem_raw[];
    __shared__ int s_dead;
    __shared__ uint32_t s_tmem;
    const int split = blockIdx.z, splits = KV ? a.splits_kv : a.splits_q;
    if (split >= splits) return;
    const AttnTile tl = KV ? attn_tile<B::kOwn>(a.k_off, a.q_off, a.graphs, 1, tile) : attn_tile<B::kOwn>(a.q_off, a.k_off, a.graphs, a.group, tile);
    if (tl.graph < 0) return;
    const int64_t q0 = KV ? tl.other : tl.first, k0 = KV ? tl.first : tl.other;
    const int64_t rows = KV ? tl.n * a.group : tl.rows, states = KV ? tl.rows : tl.n;
    const Piece walk = piece_of(KV ? rows : states, split, splits);
    const int n_tiles = uniform(int((walk.hi - walk.lo + B::kWalk - 1) / B::kWalk));
    const int own = int(min(tl.rows - tl.row0, int64_t(B::kOwn)));
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = uniform(smem_u32(smem));
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t r_full = sb + B::kBars, s_full = r_full + 8, dp_full = s_full + 8, p_ready = dp_full + 8, ds_ready = p_ready + 8,
                   done = ds_ready + 8, fin = done + 8, full = fin + 8, empty = full + 8 * B::kStages, aux_full = empty + 8 * B::kStages;
    if (threadIdx.x == 0) {
        s_dead = 0;
        bar_init(r_full, kLoadThreads);
        bar_init(s_full, 1);
        bar_init(dp_full, 1);
        bar_init(p_ready, B::kWarps);
        bar_init(ds_ready, B::kWarps);
        bar_init(done, 1);
        bar_init(fin, 1);
        for (int s = 0; s < B::kStages; ++s) {
            bar_init(full + 8 * s, kLoadThreads);
            bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < B::kHalfRing; ++s) bar_init(aux_full + 8 * s, kLoadThreads);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == B::kWarps) tmem_alloc(smem_u32(&s_tmem), B::kColumns);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(&s_tmem));
    volatile int* dead = &s_dead;
    unsigned* status = &attn_status_word;

    if (warp < B::kWarps) {
        // ----------------------------------------------------------------- P and dS
        const int w = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const bool work = quad * 32 < own;
        const uint32_t base_t = tmem + (uint32_t(quad * 32) << 16);
        const float c = a.scale_log2;
        const int64_t p = tl.row0 + row;
        float lse = -INFINITY, delta = 0.f;  // minus the thread's row's (dq)
        int64_t rh = 0;
        bool keep = row < own;
        if (keep) {
            if (KV) {
                rh = (k0 + p) * a.Hkv + h;
                keep = !a.keep || a.keep[k0 + p];
            } else {
                rh = (q0 + p / a.group) * a.Hq + int64_t(h) * a.group + p % a.group;
                const float v = a.lse[rh];
                lse = v == -INFINITY ? -INFINITY : -v * kLog2e;  // a row without a kept state: P = exp2(s - inf) = 0 ...
                keep = v != -INFINITY;                           // ... and a zero gradient, whatever q and d_out hold
                delta = -a.delta[rh];
            }
        }
        const int64_t n = KV ? a.nk * a.Hkv : a.nq * a.Hq;
        const int c0 = KV ? 0 : w * kCols;
        // dk (0) or dv (1), or dq
        auto gradient = [&](int which) {
            if (splits > 1) return (KV ? a.part_kv : a.part_q) + ((KV && which ? splits + split : split) * n + rh) * a.D;
            return static_cast<float*>(KV ? (which ? a.dv : a.dk) : a.dq) + rh * a.D;
        };
        auto columns = [&](int which) { return base_t + B::kG + (KV ? which * B::kGrad : w * kCols); };
        float acc[B::kHeld ? 1 : kCols];
        if constexpr (!B::kHeld) {
#pragma unroll
            for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
        }
        // What tensor memory has summed before step j (all of it: its last product is complete), small terms first: into
        // registers after every step, or into the gradient after kFlush.
        auto take = [&](int which, int j) {
            if (j == 0) return;
            if constexpr (!B::kHeld) {
                add_columns<kCols, PS, 2>(columns(which), acc);
            } else if (j % B::kFlush == 0 || j == n_tiles) {
                const float scale = KV && which ? 1.f : a.scale;
#pragma unroll 1
                for (int b = 0; b < kCols / 16; ++b) {
                    float o[16], small[16];
                    __syncwarp();
                    tmem_ld16(columns(which) + 16 * b, o);
                    if constexpr (!B::kTogether) {
                        tmem_ld16(columns(which) + PS + 16 * b, small);
                        tmem_wait_ld(small);
                    }
                    tmem_wait_ld(o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = keep ? (B::kTogether ? o[i] : o[i] + small[i]) : 0.f;
                    if (row < own) store_row<16>(gradient(which), o, scale, c0 + 16 * b, a.D, j > B::kFlush);
                }
            }
        };
        const bool tail = (walk.hi - walk.lo) % B::kWalk != 0;
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
            const int ax = j % B::kHalfRing;
            const float* s_lse = reinterpret_cast<const float*>(smem + B::kAux + ax * B::kAuxBytes) + B::kHalf * w;
            const float* s_delta = s_lse + B::kWalk;
            const bool biased = !KV && (a.keep || (tail && j == n_tiles - 1));
            if (KV || biased) {
                ok = warp_wait(aux_full + 8 * ax, a.keep || KV ? (j / B::kHalfRing) & 1 : 0, dead, status);
                if (!ok) break;
            }
            ok = warp_wait(s_full, j & 1, dead, status);
            if (!ok) break;
            fence_after();
            float v[B::kHalf];
            if (work) {
                if (KV && (B::kGroups == 1 || w == 1)) take(1, j);  // dv of the step before is complete when S of this one is
                load_columns(base_t + B::kHalf * w, v);
                tmem_wait_ld(v);
                if (biased) add_bias(v, s_lse);
                bwd_p<KV>(v, F2(c, c), lse, s_lse);
                if (KV) {
                    store_planes(v, base_t + B::kHalf * w, base_t + B::kP1 + B::kHalf / 2 * w, base_t + B::kP2 + B::kHalf / 2 * w);
                    tmem_wait_st();
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_ready);
            ok = warp_wait(dp_full, j & 1, dead, status);
            if (!ok) break;
            fence_after();
            if (work) {
                if (!KV || w == 0) take(0, j);  // dk, dq of the step before: complete when dP of this one is
                float y[B::kHalf];
                load_columns(base_t + B::kDp + B::kHalf * w, y);
                tmem_wait_ld(y);
                bwd_ds<KV>(y, v, F2(1.f, 1.f), delta, s_delta);
                store_planes(y, base_t + B::kDp + B::kHalf * w, base_t + B::kD1 + B::kHalf / 2 * w,
                             base_t + B::kD2 + B::kHalf / 2 * w);
                tmem_wait_st();
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(ds_ready);
        }
        if (ok && n_tiles > 0) {
            ok = warp_wait(done, 0, dead, status);
            fence_after();
        }
        if (ok && work) {
            // dk, dv: warpgroup 0 and 1, or one after the other by the only one
#pragma unroll 1
            for (int which = w; which < (KV ? 2 : w + 1); which += B::kGroups) {
                const int at = KV ? which : 0;
                take(at, n_tiles);
                if constexpr (!B::kHeld) {
                    if (!keep) {
#pragma unroll
                        for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
                    }
                    if (row < own) store_row<kCols>(gradient(at), acc, KV && at ? 1.f : a.scale, c0, a.D);
                } else if (n_tiles == 0 && row < own) {
                    const float none[16] = {};
                    for (int b = 0; b < kCols / 16; ++b) store_row<16>(gradient(at), none, 0.f, c0 + 16 * b, a.D);
                }
            }
        }
    } else if (warp == B::kWarps) {
        // ----------------------------------------------------------------- matrix instructions
        {
            const uint32_t lead = elect_lane();
            const uint32_t id_s = mma_desc<__nv_bfloat16>(B::kWalk, false), id2 = mma_desc<__nv_bfloat16>(2 * PS, true),
                           id1 = mma_desc<__nv_bfloat16>(PS, true);
            const uint32_t r1 = sb, r2 = sb + uint32_t(B::kTile);
            auto stage = [&](int i) { return sb + uint32_t(B::kRing + (i % B::kStages) * B::kStep); };
            auto wait_stage = [&](int i) {
                if (!warp_wait(full + 8 * (i % B::kStages), (i / B::kStages) & 1, dead, status)) return false;
                fence_async();
                return true;
            };
            auto product = [&](uint32_t d, uint32_t r, uint32_t xs, uint32_t bar) {
                six_products<PS>(lead, d, r, B::kOwnPanel, xs, B::kPanel, id_s);
                mma_commit(lead, bar);
            };
            // d = A X over the step's rows, or d += A X (not `fresh`), A in planes at a0 (its warpgroups' halves apart), a1, a2:
            // P0 X0 into PS columns, the small terms into PS more
            auto sum = [&](uint32_t d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t xs, bool fresh) {
                auto block = [&](int q, int s) { return q == 0 ? a0 + block_column(s, B::kHalf) : (q == 1 ? a1 : a2) + 8 * s; };
#pragma unroll
                for (int s = 0; s < B::kWalk / 16; ++s) {
                    auto x = [&](int plane) { return desc_rows(xs, s, B::kPanel, plane * PS); };
                    const uint32_t small = d + (B::kTogether ? 0 : PS);
                    if constexpr (B::kTogether) {
                        mma_ts(lead, d, block(0, s), x(0), id1, !fresh || s > 0);
                        mma_ts(lead, d, block(0, s), x(1), id1, true);
                    } else {
                        mma_ts(lead, d, block(0, s), x(0), id2, !fresh || s > 0);  // [X0 | X1]
                    }
                    mma_ts(lead, small, block(0, s), x(2), id1, true);
                    mma_ts(lead, small, block(1, s), x(0), id1, true);
                    mma_ts(lead, small, block(1, s), x(1), id1, true);
                    mma_ts(lead, small, block(2, s), x(0), id1, true);
                }
            };
            auto fresh = [](int j) { return !B::kHeld || j % B::kFlush == 0; };
            bool ok = n_tiles > 0 && warp_wait(r_full, 0, dead, status) && wait_stage(0);
            if (ok) {
                product(tmem, r1, stage(0), s_full);
                ok = wait_stage(1);
                if (ok) {
                    product(tmem + B::kDp, r2, stage(1), dp_full);
                    if (!KV) mma_commit(lead, empty + 8 * 1);
                }
            }
            for (int j = 0; j < n_tiles && ok; ++j) {
                ok = warp_wait(p_ready, j & 1, dead, status);
                if (!ok) break;
                fence_after();
                if (KV) {
                    sum(tmem + B::kG + B::kGrad, tmem, tmem + B::kP1, tmem + B::kP2, stage(2 * j + 1), fresh(j));
                    mma_commit(lead, empty + 8 * ((2 * j + 1) % B::kStages));
                }
                if (j + 1 < n_tiles) {
                    ok = wait_stage(2 * j + 2);
                    if (!ok) break;
                    product(tmem, r1, stage(2 * j + 2), s_full);
                }
                ok = warp_wait(ds_ready, j & 1, dead, status);
                if (!ok) break;
                fence_after();
                sum(tmem + B::kG, tmem + B::kDp, tmem + B::kD1, tmem + B::kD2, stage(2 * j), fresh(j));
                mma_commit(lead, empty + 8 * ((2 * j) % B::kStages));
                if (j + 1 < n_tiles) {
                    ok = wait_stage(2 * j + 3);
                    if (!ok) break;
                    product(tmem + B::kDp, r2, stage(2 * j + 3), dp_full);
                    if (!KV) mma_commit(lead, empty + 8 * ((2 * j + 3) % B::kStages));
                } else {
                    mma_commit(lead, done);
                }
            }
            mma_commit(lead, fin);
            bar_wait_last(fin, 0, status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------------- loaders
        const int t = threadIdx.x - (B::kWarps + 1) * 32;
        if (n_tiles > 0) {
            constexpr int64_t kHead = 3 * PS * 2;  // bytes of a (row, head)
            const int64_t q_at = (q0 * a.Hq + int64_t(h) * a.group) * kHead, q_row = a.Hq * kHead, k_row = a.Hkv * kHead;
            const char *Q = reinterpret_cast<const char*>(x.q) + q_at, *dO = reinterpret_cast<const char*>(x.d_out) + q_at;
            const int64_t k_at = ((k0 + (KV ? tl.row0 : walk.lo)) * a.Hkv + h) * kHead;
            const char *K = reinterpret_cast<const char*>(x.k) + k_at, *V = reinterpret_cast<const char*>(x.v) + k_at;
            auto free_stage = [&](int i) {
                return i < B::kStages || warp_wait(empty + 8 * (i % B::kStages), (i / B::kStages - 1) & 1, dead, status);
            };
            auto stage = [&](int i) { return sb + uint32_t(B::kRing + (i % B::kStages) * B::kStep); };
            if (KV) {
                StateMask<B::kOwn> mask(a.keep ? a.keep + k0 : nullptr, tl.row0, states);
                mask.next();
                load_planes<PS>(sb, K, k_row, t, mask);
                load_planes<PS>(sb + uint32_t(B::kTile), V, k_row, t, mask);
            } else {
                load_planes_packed<PS, B::kOwn, false>(sb, Q, q_row, kHead, a.group, tl.row0, own, t);
                load_planes_packed<PS, B::kOwn, false>(sb + uint32_t(B::kTile), dO, q_row, kHead, a.group, tl.row0, own, t);
            }
            copy_arrive(r_full);
            // lse and delta of the walked rows, fetched a step ahead
            float v_lse = -INFINITY, v_delta = 0.f;
            RowWalk stats(walk.lo + t, a.group, q0 * a.Hq + int64_t(h) * a.group, a.Hq, B::kWalk);
            auto fetch = [&]() {
                v_lse = -INFINITY, v_delta = 0.f;
                if (t < B::kWalk && stats.r < walk.hi) {
                    v_lse = a.lse[stats.at];
                    v_delta = a.delta[stats.at];
                }
                stats.next();
            };
            if (KV) fetch();
            StateMask<B::kWalk> mask(!KV && a.keep ? a.keep + k0 : nullptr, walk.lo, walk.hi);
            for (int j = 0; j < n_tiles; ++j) {
                const int64_t lo = walk.lo + int64_t(j) * B::kWalk;
                const int n = int(min(walk.hi - lo, int64_t(B::kWalk)));
                if (!free_stage(2 * j)) break;
                // the step that used this aux entry before gave up its X1 stage, which is this one
                if (KV) {
                    float* s_lse = reinterpret_cast<float*>(smem + B::kAux + (j % B::kHalfRing) * B::kAuxBytes);
                    // rows past the end and rows without a kept state: P = exp2(s - inf) = 0
                    if (t < B::kWalk) {
                        s_lse[t] = v_lse == -INFINITY ? -INFINITY : -v_lse * kLog2e;
                        s_lse[B::kWalk + t] = -v_delta;
                    }
                    bar_arrive(aux_full + 8 * (j % B::kHalfRing));
                    if (j + 1 < n_tiles) fetch();
                    load_planes_packed<PS, B::kWalk, true>(stage(2 * j), Q, q_row, kHead, a.group, lo, n, t);
                    copy_arrive(full + 8 * ((2 * j) % B::kStages));
                    if (!free_stage(2 * j + 1)) break;
                    load_planes_packed<PS, B::kWalk, true>(stage(2 * j + 1), dO, q_row, kHead, a.group, lo, n, t);
                    copy_arrive(full + 8 * ((2 * j + 1) % B::kStages));
                } else {
                    mask.next();
                    if (a.keep || n < B::kWalk) {
                        write_bias(reinterpret_cast<float*>(smem + B::kAux + (j % B::kHalfRing) * B::kAuxBytes), mask, t);
                        bar_arrive(aux_full + 8 * (j % B::kHalfRing));
                    }
                    load_planes<PS>(stage(2 * j), K, k_row, t, mask);
                    copy_arrive(full + 8 * ((2 * j) % B::kStages));
                    if (!free_stage(2 * j + 1)) break;
                    load_planes<PS>(stage(2 * j + 1), V, k_row, t, mask);
                    copy_arrive(full + 8 * ((2 * j + 1) % B::kStages));
                    K += B::kWalk * k_row;
                    V += B::kWalk * k_row;
                }
            }
            copy_wait_all();
        }
    }
    fence_before();
    __syncthreads();
    if (warp == B::kWarps) {
        fence_after();
        tmem_free(tmem, B::kColumns);
    }
}

template <int PS>
constexpr int kBwdThreads = (BwdPlan<PS, true>::kWarps + 1 + kLoadWarps) * 32;

template <int PS>
__global__ void __launch_bounds__(kBwdThreads<PS>, BwdPlan<PS, true>::kColumns == 256 ? 2 : 1)
    attn_bwd_planes(const __grid_constant__ AttnArgs a, Planes x) {
    const BwdTile t = bwd_tile_of(a);
    if (t.kv)
        bwd_tile<PS, true>(a, x, t.tile, t.head);
    else
        bwd_tile<PS, false>(a, x, t.tile, t.head);
}

template <typename F>
cudaError_t by_plane(int D, F f) {
    if (D <= 16) return f(std::integral_constant<int, 16>{});
    if (D <= 32) return f(std::integral_constant<int, 32>{});
    if (D <= 64) return f(std::integral_constant<int, 64>{});
    return f(std::integral_constant<int, 128>{});
}
int plane_stride(int D) { return D <= 16 ? 16 : D <= 32 ? 32 : D <= 64 ? 64 : 128; }

// The planes' places in the workspace, in the order q, k, v, d_out.
Planes planes_at(const AttnArgs& a, void* ws) {
    const size_t w = size_t(3) * plane_stride(a.D);
    uint16_t* p = static_cast<uint16_t*>(ws);
    Planes x;
    x.q = p;
    x.k = x.q + size_t(a.nq) * a.Hq * w;
    x.v = x.k + size_t(a.nk) * a.Hkv * w;
    x.d_out = x.v + size_t(a.nk) * a.Hkv * w;
    return x;
}

}  // namespace

size_t attn_planes_bytes(const AttnShape& s, bool bwd) {
    const size_t w = size_t(6) * plane_stride(s.head_dim);
    const size_t q = size_t(s.n_q) * s.q_heads * w, k = size_t(s.n_k) * s.kv_heads * w;
    return q + 2 * k + (bwd ? q : 0);
}

cudaError_t launch_attn_planes(const AttnArgs& a, void* ws, int sms, cudaStream_t st) {
    const Planes x = planes_at(a, ws);
    const auto vec = [&](const void* p, int64_t row, int64_t head) {
        return a.D % 4 == 0 && row % 4 == 0 && head % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
    };
    const auto job = [&](const void* p, int64_t row, int64_t head, int64_t rows, int heads, const uint16_t* out) {
        return PlaneJob{static_cast<const float*>(p), row, head, rows, heads, const_cast<uint16_t*>(out), vec(p, row, head)};
    };
    PlaneJobs j = {};
    j.D = a.D;
    j.j[0] = job(a.q, a.q_row, a.q_head, a.nq, a.Hq, x.q);
    j.j[1] = job(a.k, a.k_row, a.k_head, a.nk, a.Hkv, x.k);
    j.j[2] = job(a.v, a.v_row, a.v_head, a.nk, a.Hkv, x.v);
    const bool bwd = a.delta != nullptr;
    if (bwd) {
        j.j[3] = job(a.d_out, a.o_row, a.o_head, a.nq, a.Hq, x.d_out);
        j.vec_o = j.j[3].vec && vec(a.out, a.o_row, a.o_head);
    }
    const unsigned blocks = unsigned(std::min<int64_t>((std::max(a.nq, a.nk) + 63) / 64, int64_t(sms) * 8));
    return by_plane(a.D, [&](auto ps) {
        attn_planes<decltype(ps)::value><<<dim3(blocks, bwd ? 5 : 3), 256, 0, st>>>(j, a);
        return cudaGetLastError();
    });
}

cudaError_t launch_attn_fwd_planes(const AttnArgs& a, void* ws, int64_t row_tiles, cudaStream_t st) {
    const Planes x = planes_at(a, ws);
    return by_plane(a.D, [&](auto ps) {
        constexpr int PS = decltype(ps)::value;
        using F = FwdPlan<PS>;
        cudaError_t e = cudaFuncSetAttribute(attn_fwd_planes<PS>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kTotal);
        if (e != cudaSuccess) return e;
        attn_fwd_planes<PS><<<dim3(unsigned(row_tiles), unsigned(a.Hkv), unsigned(a.splits)), F::kThreads, F::kTotal, st>>>(a, x);
        return cudaGetLastError();
    });
}

cudaError_t launch_attn_bwd_planes(const AttnArgs& a, void* ws, cudaStream_t st) {
    const Planes x = planes_at(a, ws);
    return by_plane(a.D, [&](auto ps) {
        constexpr int PS = decltype(ps)::value;
        constexpr int smem = std::max(BwdPlan<PS, true>::kTotal, BwdPlan<PS, false>::kTotal);
        cudaError_t e = cudaFuncSetAttribute(attn_bwd_planes<PS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        attn_bwd_planes<PS><<<bwd_grid(a), kBwdThreads<PS>, smem, st>>>(a, x);
        return cudaGetLastError();
    });
}

cudaError_t attn_planes_status(unsigned* word, bool reset) { return read_status(word, reset); }

}  // namespace uvu
