// The attention backward on the tensor cores for 16-bit operands.
//
// KV false: dq of a tile of 128 packed rows, walking the states; KV true: dk and dv of a tile of 128
// states, walking the packed rows of all heads that share them (so a shared head's gradient needs no
// second sum).  R1, R2: the tile's own operands, resident; X1, X2: the walked ones, in the ring.
//              R1  R2  X1  X2      S = R1 X1^T,  dP = R2 X2^T,  P = exp2(c S - lse),  dS = P (dP - delta)
//     dq       Q   dO  K   V       dq += dS X1
//     dk, dv   K   V   Q   dO      dk += dS X1,  dv += P X2      (S and dP transposed: lanes are states)
// Both kinds of tile are in one launch.  Two sweeps instead of one cost S and dP twice (seven products instead of five),
// but every sum stays in one CTA's tensor memory: no atomics, and results that do not depend on timing.  Long
// walks take their sums out of tensor memory on the way (attn_hold_tiles), to fp32 values that the join rounds.
//
// Tensor memory: S, dP (128 columns each), then the sums.  P and dS are written as 16-bit values over
// the part of S and dP that the same thread has read.  Two warpgroups share a tile: warpgroup w takes
// columns 64 w .. + 63 of each lane's row.  Order of the matrix instructions:
//     S(0) dP(0) | dv += P(0) X2, S(1), dk += dS(0) X1, dP(1) | ...
// so the tensor cores form dv(j) and S(j+1) while the threads turn dP(j) into dS(j), and dk(j) and
// dP(j+1) while they turn S(j+1) into P(j+1).  (A second S, to head dimension 64 where columns are left for it: 1757
// against 1733 us for 16 heads of 64 at 4 x 4096 rows and states, forward and backward.)
//
// Measured, 16 heads at 4 x 4096 rows and states: dq 489 us, dk and dv 643 us at head dimension 64; 724 and 855 at 128 (a
// third to a half of the tensor cores' time).  Bound: the threads' P and dS (64 exponentials a thread and step at 8 a clock
// and quarter of an SM) and the hand-overs between them and the issuing warp, some 700 clocks each.  Half tiles handed over one
// warpgroup at a time were slower (639 and 695 us at 64).
//
// P and dS are rounded to the operands' type for their products, which take no other; the sums are fp32.  delta comes from the rounded
// output: d_q of a bf16 batch is off by 2.6e-3 (relative) where its own rounding gives 1.7e-3.
// bf16 has the exponent range of fp32.  f16 does not, so its P and dS are held at a scale, undone in the epilogue:
//   - 2^8 P (for dv): P of long rows would fall below the type's smallest normal value, 2^-14.
//   - 2^e dS: |dS| <= 2 P |do| max_j |v_j| follows the cotangent's size.  e puts this bound at most at 2^15: nothing overflows, and
//     dS keeps its bits down to 2^-29 of the bound.  A row of dq has its own |do|; dk sums over rows and takes the largest of
//     the graph's rows and the kv head's heads.  Squares and maxima come with delta (attn.cu), for 2.5% of the backward: 8 graphs
//     to 4096 rows, 16/4 heads of 64, 1045 -> 1073 us; 3 us of the smallest.  dq over 4096 states is off by 6.9e-4 with cotangents of
//     size 1e-3 (its own rounding: 6.5e-4) and would be by 5.2e-3 with dS at no scale, since 2^-14 is far above it.
#include "attn_mma.h"

namespace uvu {
namespace {

template <bool KV>
struct BwdLayout {
    int panels, log_stages, stages;  // a power of two: a division by a variable costs the issuer as much as several instructions
    __device__ int at(int i) const { return i & (stages - 1); }               // of the ring's use i: its stage,
    __device__ uint32_t parity(int i) const { return (i >> log_stages) & 1; }  // its phase
    __host__ __device__ int tile() const { return panels * kPanelBytes; }
    __host__ __device__ int ring() const { return 2 * tile(); }
    __host__ __device__ int aux() const { return ring() + stages * tile(); }  // per walked tile: -lse and -delta, or the states' bias
    __host__ __device__ int aux_bytes() const { return (KV ? 2 : 1) * kRows * 4; }
    __host__ __device__ int bars() const { return aux() + stages / 2 * aux_bytes(); }
    __host__ __device__ int total() const { return bars() + 256 + 1024; }  // + alignment slack
};

// Four warps that load: with two, dk and dv of 16 heads of 64 at 4 x 4096 rows and states took 792 us instead of 723 (and the
// forward, whose softmax needs the registers, 720 instead of 400 with four).
constexpr int kBwdLoad = 4 * 32, kBwdWarps = 8 + 1 + kBwdLoad / 32;

// e of the scale 2^e of dS: 2 |do| |v| 2^e <= 2^15, from the squares' product below 2^(x + 1).  Without a bound (an operand that
// is not finite) or without a value the scale is 1.
__device__ __forceinline__ int ds_exponent(float do2, float v2) {
    const float b = do2 * v2;
    if (!(b > 0.f) || b == INFINITY) return 0;
    const int x = int(__float_as_uint(b) >> 23) - 127;
    return 14 - ((x + 2) >> 1);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// 16 columns of a gradient row, times `scale`, to a partial or final row of D values.
template <typename T>
__device__ __forceinline__ void store_grad16(const float (&o)[16], float scale, T* dst, float* part, int c0, int D, bool vec) {
    if (part) {
        if (D % 4 == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c0 + 4 * i < D)
                    *reinterpret_cast<float4*>(part + c0 + 4 * i) =
                        make_float4(o[4 * i] * scale, o[4 * i + 1] * scale, o[4 * i + 2] * scale, o[4 * i + 3] * scale);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c0 + i < D) part[c0 + i] = o[i] * scale;
        }
    } else if (vec) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (c0 + 8 * i < D)
                *reinterpret_cast<uint4*>(dst + c0 + 8 * i) =
                    make_uint4(pack2<T>(o[8 * i] * scale, o[8 * i + 1] * scale), pack2<T>(o[8 * i + 2] * scale, o[8 * i + 3] * scale),
                               pack2<T>(o[8 * i + 4] * scale, o[8 * i + 5] * scale), pack2<T>(o[8 * i + 6] * scale, o[8 * i + 7] * scale));
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (c0 + i < D) dst[c0 + i] = narrow<T>(o[i] * scale);
    }
}

// Adds every `step`-th 16 columns of a row's sums from d on to what a long walk holds of them (null: a lane without a gradient).
static __device__ __noinline__ void hold_sums(uint32_t sums, int d, int step, int d16, int D, float* held, float scale, bool first) {
    for (; d < d16; d += step) {
        float o[16];
        __syncwarp();
        tmem_ld16(sums + 16 * d, o);
        tmem_wait_ld(o);
        if (!held) continue;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (16 * d + i < D) held[16 * d + i] = fmaf(o[i], scale, first ? 0.f : held[16 * d + i]);
    }
}

template <typename T, int LG, bool ALIGNED, bool HELD, bool KV>
__device__ __forceinline__ void bwd_tile(const AttnArgs& a, const BwdLayout<KV>& L, int64_t tile, int h) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ int s_dead;
    __shared__ uint32_t s_tmem;
    const int split = blockIdx.z, splits = KV ? a.splits_kv : a.splits_q;
    if (split >= splits) return;
    const AttnTile tl = KV ? attn_tile<kRows>(a.k_off, a.q_off, a.graphs, 1, tile) : attn_tile<kRows>(a.q_off, a.k_off, a.graphs, a.group, tile);
    if (tl.graph < 0) return;
    const int64_t q0 = KV ? tl.other : tl.first, k0 = KV ? tl.first : tl.other;
    const int64_t rows = KV ? tl.n * a.group : tl.rows, states = KV ? tl.rows : tl.n;
    const Piece walk = piece_of(KV ? rows : states, split, splits);
    const int n_tiles = uniform(int((walk.hi - walk.lo + kRows - 1) / kRows));
    const int own = int(min(tl.rows - tl.row0, int64_t(kRows)));  // rows of the resident tile
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = uniform(smem_u32(smem));
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int d16 = (a.D + 15) / 16, half = L.stages / 2;
    const uint32_t r_full = sb + L.bars(), s_full = r_full + 8, dp_full = s_full + 8, p_ready = dp_full + 8, ds_ready = p_ready + 8,
                   done = ds_ready + 8, fin = done + 8, full = fin + 8, empty = full + 8 * L.stages, aux_full = empty + 8 * L.stages;
    const uint32_t g_cols = uint32_t(64 * L.panels);
    const uint32_t tmem_cols = 512;
    if (threadIdx.x == 0) {
        s_dead = 0;
        bar_init(r_full, kBwdLoad);
        bar_init(s_full, 1);
        bar_init(dp_full, 1);
        bar_init(p_ready, 8);
        bar_init(ds_ready, 8);
        bar_init(done, 1);
        bar_init(fin, 1);
        for (int s = 0; s < L.stages; ++s) {
            bar_init(full + 8 * s, kBwdLoad);
            bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < half; ++s) bar_init(aux_full + 8 * s, kBwdLoad);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) tmem_alloc(smem_u32(&s_tmem), tmem_cols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(&s_tmem));
    const uint32_t t_dp = tmem + kRows, t_g = tmem + 2 * kRows;  // sums: dq, or dk then dv
    volatile int* dead = &s_dead;
    unsigned* status = &attn_status_word;
    constexpr bool kScaled = __is_same(T, __half);
    constexpr float kShift = kScaled ? 8.f : 0.f, kUnshift = kScaled ? 0.00390625f : 1.f;
    // the exponent of dS's scale: (2^8 P) (dP u - delta u) with u = 2^(e - 8) for dk, (2^e P) (dP - delta) for dq
    auto exponent = [&](float do2) { return ds_exponent(do2, __uint_as_float(a.v2_top[int64_t(tl.graph) * a.Hkv + h])); };
    auto tile_exponent = [&]() {  // of dk: the same for the whole tile
        return kScaled && n_tiles > 0 ? exponent(__uint_as_float(a.do2_top[int64_t(tl.graph) * a.Hkv + h])) : 0;
    };
    constexpr float kLog2e = 1.4426950408889634f;
    // the sums begin anew at these tiles
    float* const parts = KV ? a.part_kv : a.part_q;
    constexpr int kHold = attn_hold_tiles(kScaled);
    const bool held = HELD && parts && n_tiles > kHold;
    auto fresh = [&](int j) { return j == 0 || (HELD && held && j % kHold == 0); };

    if (warp < 8) {
        // ----------------------------------------------------------------- P and dS
        const int w = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const bool work = quad * 32 < own;
        const uint32_t lanes = uint32_t(quad * 32) << 16, col = uint32_t(64 * w);
        const float c = a.scale_log2;
        const int64_t p = tl.row0 + row;
        float lse = -INFINITY, delta = 0.f;  // minus the thread's row's (dq)
        int64_t rh = 0;
        int e_ds = KV ? tile_exponent() : 0;
        bool keep = row < own;
        if (keep) {
            if (KV) {
                rh = (k0 + p) * a.Hkv + h;
                keep = !a.keep || a.keep[k0 + p];
            } else {
                rh = (q0 + p / a.group) * a.Hq + int64_t(h) * a.group + p % a.group;
                const float x = a.lse[rh];
                if (kScaled) e_ds = exponent(a.do2[rh]);
                // P is not stored here, so dS's scale is its own.  A row without a kept state: P = exp2(s - inf) = 0, and a
                // zero gradient, whatever q and d_out hold
                lse = x == -INFINITY ? -INFINITY : float(e_ds) - x * kLog2e;
                keep = x != -INFINITY;
                delta = -a.delta[rh];
            }
        }
        const float u = KV ? kUnshift * power_of_two(e_ds) : 1.f;
        // the thread's gradient row, dk: warpgroup 0, dv: warpgroup 1
        const int64_t n_grads = KV ? a.nk * a.Hkv : a.nq * a.Hq;
        auto part_row = [&]() { return parts + ((KV && w ? splits + split : split) * n_grads + rh) * a.D; };
        const float grad_scale = KV && w ? kUnshift : a.scale * power_of_two(-e_ds);
        auto hold = [&](int j) {
            hold_sums(t_g + lanes + (KV ? uint32_t(w) * g_cols : 0u), KV ? 0 : w, KV ? 1 : 2, d16, a.D, row < own && keep ? part_row() : nullptr,
                      grad_scale, j == kHold);
        };
        const bool tail = (walk.hi - walk.lo) % kRows != 0;
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
            const int ax = j & (half - 1);
            const float* s_lse = reinterpret_cast<const float*>(smem + L.aux() + ax * L.aux_bytes()) + col;  // or the bias
            const float* s_delta = s_lse + kRows;
            const bool biased = !KV && (a.keep || (tail && j == n_tiles - 1));
            if (KV || biased) {
                ok = warp_wait(aux_full + 8 * ax, a.keep || KV ? L.parity(2 * j) : 0, dead, status);
                if (!ok) break;
            }
            ok = warp_wait(s_full, j & 1, dead, status);
            if (!ok) break;
            fence_after();
            float x[2][32];
            if (work) {
                if (HELD && KV && w == 1 && j > 0 && fresh(j)) hold(j);  // dv of the tile before is complete when S of this one is
#pragma unroll
                for (int b = 0; b < 2; ++b) tmem_ld32(tmem + lanes + col + 32 * b, x[b]);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    tmem_wait_ld(x[b]);
                    if (biased) add_bias(x[b], s_lse + 32 * b);
                    bwd_p<KV>(x[b], F2(c, c), lse, s_lse + 32 * b);
                    if (KV) {
                        uint32_t q[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) q[i] = pack2<T>(x[b][2 * i], x[b][2 * i + 1]);
                        tmem_st16(tmem + lanes + col + 16 * b, q);
                    }
                }
                if (KV) tmem_wait_st();
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(p_ready);
            ok = warp_wait(dp_full, j & 1, dead, status);
            if (!ok) break;
            fence_after();
            if (work) {
                if (HELD && !(KV && w == 1) && j > 0 && fresh(j)) hold(j);  // dk, dq: when dP of this one is
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float y[32];
                    tmem_ld32(t_dp + lanes + col + 32 * b, y);
                    tmem_wait_ld(y);
                    bwd_ds<KV>(y, x[b], F2(u, u), delta, s_delta + 32 * b);
                    uint32_t q[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) q[i] = pack2<T>(y[2 * i], y[2 * i + 1]);
                    tmem_st16(t_dp + lanes + col + 16 * b, q);
                }
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
            // dq: the column blocks in turn
            T* dst = static_cast<T*>(KV ? (w ? a.dv : a.dk) : a.dq) + rh * a.D;
            float* part = parts ? part_row() : nullptr;
            const bool vec = a.D % 8 == 0 && (reinterpret_cast<uintptr_t>(dst) & 15u) == 0;
            for (int d = KV ? 0 : w; d < d16; d += KV ? 1 : 2) {
                float o[16];
                __syncwarp();
                if (n_tiles > 0) {
                    tmem_ld16(t_g + lanes + (KV ? uint32_t(w) * g_cols : 0u) + 16 * d, o);
                    tmem_wait_ld(o);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = n_tiles > 0 && keep ? o[i] : 0.f;
                if (HELD && held && row < own && keep) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (16 * d + i < a.D) part[16 * d + i] = fmaf(o[i], grad_scale, part[16 * d + i]);
                } else if (row < own) {
                    store_grad16<T>(o, grad_scale, dst, part, 16 * d, a.D, vec);
                }
            }
        }
    } else if (warp == 8) {
        // ----------------------------------------------------------------- matrix instructions
        {
            const uint32_t lead = elect_lane();
            const uint32_t id_s = mma_desc<T>(kRows, false), id_g = mma_desc<T>(16 * d16, true);
            const uint32_t r1 = sb, r2 = sb + uint32_t(L.tile());
            auto stage = [&](int i) { return sb + uint32_t(L.ring() + L.at(i) * L.tile()); };
            auto wait_stage = [&](int i) {
                if (!warp_wait(full + 8 * L.at(i), L.parity(i), dead, status)) return false;
                fence_async();
                return true;
            };
            auto product = [&](uint32_t d, uint32_t r, uint32_t x, uint32_t bar) {
#pragma unroll
                for (int s = 0; s < 1 << (LG - 1); ++s)  // all of them, or fewer off the class's largest head dimension
                    if (s < d16) mma_ss(lead, d, desc_cols(r, s), desc_cols(x, s), id_s, s > 0);
                mma_commit(lead, bar);
            };
            // d += A X: the 16-bit A of row block s lies in the half that its warpgroup wrote
            auto sum = [&](uint32_t d, uint32_t A, uint32_t x, bool first) {
#pragma unroll
                for (int s = 0; s < kRows / 16; ++s)
                    mma_ts(lead, d, A + uint32_t((s >> 2) * 64 + (s & 3) * 8), desc_rows(x, s), id_g, !first || s > 0);
            };
            bool ok = n_tiles > 0 && warp_wait(r_full, 0, dead, status) && wait_stage(0);
            if (ok) {
                product(tmem, r1, stage(0), s_full);
                ok = wait_stage(1);
                if (ok) {
                    product(t_dp, r2, stage(1), dp_full);
                    if (!KV) mma_commit(lead, empty + 8 * 1);
                }
            }
            for (int j = 0; j < n_tiles && ok; ++j) {
                ok = warp_wait(p_ready, j & 1, dead, status);
                if (!ok) break;
                fence_after();
                if (KV) {
                    sum(t_g + g_cols, tmem, stage(2 * j + 1), fresh(j));
                    mma_commit(lead, empty + 8 * L.at(2 * j + 1));
                }
                if (j + 1 < n_tiles) {
                    ok = wait_stage(2 * j + 2);
                    if (!ok) break;
                    product(tmem, r1, stage(2 * j + 2), s_full);
                }
                ok = warp_wait(ds_ready, j & 1, dead, status);
                if (!ok) break;
                fence_after();
                sum(t_g, t_dp, stage(2 * j), fresh(j));
                mma_commit(lead, empty + 8 * L.at(2 * j));
                if (j + 1 < n_tiles) {
                    ok = wait_stage(2 * j + 3);
                    if (!ok) break;
                    product(t_dp, r2, stage(2 * j + 3), dp_full);
                    if (!KV) mma_commit(lead, empty + 8 * L.at(2 * j + 3));
                } else {
                    mma_commit(lead, done);
                }
            }
            // every instruction issued has finished before the tensor memory and the stages go
            mma_commit(lead, fin);
            bar_wait_last(fin, 0, status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------------- loaders
        const int t = threadIdx.x - 9 * 32;
        const LoadMap<LG, kRows, kBwdLoad> map(t, a.D);
        if (n_tiles > 0) {
            auto arrive = [&](uint32_t bar) { ALIGNED ? copy_arrive(bar) : bar_arrive(bar); };
            const char* Q = reinterpret_cast<const char*>(static_cast<const T*>(a.q) + q0 * a.q_row + int64_t(h) * a.group * a.q_head);
            const char* dO = reinterpret_cast<const char*>(static_cast<const T*>(a.d_out) + q0 * a.o_row + int64_t(h) * a.group * a.o_head);
            const int64_t s0 = k0 + (KV ? tl.row0 : walk.lo);
            const char* K = reinterpret_cast<const char*>(static_cast<const T*>(a.k) + s0 * a.k_row + h * a.k_head) + map.chunk * 16;
            const char* V = reinterpret_cast<const char*>(static_cast<const T*>(a.v) + s0 * a.v_row + h * a.v_head) + map.chunk * 16;
            StateMask<> mask(a.keep ? a.keep + k0 : nullptr, KV ? tl.row0 : walk.lo, KV ? states : walk.hi);
            auto states_tile = [&](uint32_t dst, const char* src, int64_t stride) { load_states<ALIGNED>(dst, src, stride, map, mask); };
            auto rows_tile = [&](uint32_t dst, const char* base, int64_t row, int64_t head, int64_t r0, int n) {
                load_packed<ALIGNED, KV>(dst, base, row * 2, head * 2, a.group, r0, n, map);
            };
            auto free_stage = [&](int i) {
                return i < L.stages || warp_wait(empty + 8 * L.at(i), L.parity(i - L.stages), dead, status);
            };
            auto stage = [&](int i) { return sb + uint32_t(L.ring() + L.at(i) * L.tile()); };
            if (KV) {
                mask.next();
                states_tile(sb, K, a.k_row * 2);
                states_tile(sb + uint32_t(L.tile()), V, a.v_row * 2);
            } else {
                rows_tile(sb, Q, a.q_row, a.q_head, tl.row0, own);
                rows_tile(sb + uint32_t(L.tile()), dO, a.o_row, a.o_head, tl.row0, own);
            }
            arrive(r_full);
            // lse and delta of the walked rows, fetched a tile ahead
            constexpr int kEach = kRows / kBwdLoad;
            float v_lse[kEach], v_delta[kEach];
            RowWalk stats(walk.lo + t, a.group, q0 * a.Hq + int64_t(h) * a.group, a.Hq, kBwdLoad);
            auto fetch = [&]() {
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    v_lse[i] = -INFINITY, v_delta[i] = 0.f;
                    if (stats.r < walk.hi) {
                        v_lse[i] = a.lse[stats.at];
                        v_delta[i] = a.delta[stats.at];
                    }
                    stats.next();
                }
            };
            if (KV) fetch();
            const float u = KV ? kUnshift * power_of_two(tile_exponent()) : 1.f;
            for (int j = 0; j < n_tiles; ++j) {
                const int64_t lo = walk.lo + int64_t(j) * kRows;
                const int n = int(min(walk.hi - lo, int64_t(kRows)));
                if (!free_stage(2 * j)) break;
                // the tile that used this aux entry before gave up its X1 stage, which is this one
                if (KV) {
                    float* s_lse = reinterpret_cast<float*>(smem + L.aux() + (j & (half - 1)) * L.aux_bytes());
#pragma unroll
                    for (int i = 0; i < kEach; ++i) {
                        // rows past the end and rows without a kept state: P = exp2(s - inf) = 0
                        s_lse[t + kBwdLoad * i] = v_lse[i] == -INFINITY ? -INFINITY : kShift - v_lse[i] * kLog2e;
                        s_lse[kRows + t + kBwdLoad * i] = -v_delta[i] * u;
                    }
                    bar_arrive(aux_full + 8 * (j & (half - 1)));
                    if (j + 1 < n_tiles) fetch();
                    rows_tile(stage(2 * j), Q, a.q_row, a.q_head, lo, n);
                    arrive(full + 8 * L.at(2 * j));
                    if (!free_stage(2 * j + 1)) break;
                    rows_tile(stage(2 * j + 1), dO, a.o_row, a.o_head, lo, n);
                    arrive(full + 8 * L.at(2 * j + 1));
                } else {
                    mask.next();
                    if (a.keep || n < kRows) {
                        write_bias<kBwdLoad>(reinterpret_cast<float*>(smem + L.aux() + (j & (half - 1)) * L.aux_bytes()), mask, t);
                        bar_arrive(aux_full + 8 * (j & (half - 1)));
                    }
                    states_tile(stage(2 * j), K, a.k_row * 2);
                    arrive(full + 8 * L.at(2 * j));
                    if (!free_stage(2 * j + 1)) break;
                    states_tile(stage(2 * j + 1), V, a.v_row * 2);
                    arrive(full + 8 * L.at(2 * j + 1));
                    K += kRows * a.k_row * 2;
                    V += kRows * a.v_row * 2;
                }
            }
            copy_wait_all();
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 8) {
        fence_after();
        tmem_free(tmem, tmem_cols);
    }
}

template <typename T, int LG, bool ALIGNED, bool HELD>
__global__ void __launch_bounds__(kBwdWarps * 32, 1) attn_bwd_mma(const __grid_constant__ AttnArgs a, BwdLayout<true> Lkv, BwdLayout<false> Lq) {
    const BwdTile t = bwd_tile_of(a);
    if (t.kv)
        bwd_tile<T, LG, ALIGNED, HELD, true>(a, Lkv, t.tile, t.head);
    else
        bwd_tile<T, LG, ALIGNED, HELD, false>(a, Lq, t.tile, t.head);
}

template <typename T>
cudaError_t bwd(const AttnArgs& a, cudaStream_t st) {
    BwdLayout<true> kv;
    BwdLayout<false> q;
    kv.panels = q.panels = a.D > 64 ? 2 : 1;
    kv.log_stages = q.log_stages = kv.panels == 1 ? 3 : 2;  // 160 or 192 KB
    kv.stages = q.stages = 1 << kv.log_stages;
    const uintptr_t any = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                          reinterpret_cast<uintptr_t>(a.d_out) |
                          uintptr_t(a.q_row | a.q_head | a.k_row | a.k_head | a.v_row | a.v_head | a.o_row | a.o_head) * 2;
    return by_chunks(a.D, (any & 15u) == 0, [&](auto lg, auto aligned) {
        constexpr int LG = decltype(lg)::value;
        constexpr bool ALIGNED = decltype(aligned)::value;
        auto k = a.hold ? attn_bwd_mma<T, LG, ALIGNED, true> : attn_bwd_mma<T, LG, ALIGNED, false>;
        const int smem = std::max(kv.total(), q.total());
        cudaError_t e = allow_most_smem(k, smem);
        if (e != cudaSuccess) return e;
        k<<<bwd_grid(a), kBwdWarps * 32, smem, st>>>(a, kv, q);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_attn_bwd_mma(uvu_dtype dtype, const AttnArgs& a, cudaStream_t st) {
    return dtype == UVU_BF16 ? bwd<__nv_bfloat16>(a, st) : bwd<__half>(a, st);
}

cudaError_t attn_bwd_mma_status(unsigned* word, bool reset) { return read_status(word, reset); }

}  // namespace uvu
