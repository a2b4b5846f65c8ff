// Attention on the 5th-generation tensor cores for 16-bit operands.
//
// Forward.  A CTA owns NT tiles of 128 packed rows (of one graph and kv head) and walks the graph's
// states in tiles of 128.  Per state tile j and row tile t:
//     S_t = Q_t K_j^T            (both operands in shared memory, S in tensor memory)
//     P_t = exp2(c S_t - m)      (a thread per row reads S, keeps the running maximum m and the sum of P)
//     O_t = O_t + P_t V_j        (P written over S in tensor memory as 16-bit values; V is used with its rows
//                                as the summed index, straight from the layout it was loaded in)
// The maximum that P refers to is only moved (and O_t multiplied by exp2(old - new)) when a row's new
// maximum exceeds it by more than 2^8: P <= 256 fits both 16-bit types, and nearly all tiles leave O alone.
//
// Warp roles: warps 0 .. 4 NT - 1 softmax (a warpgroup per row tile), one warp that issues the matrix
// instructions, two warps that load.  With NT = 2 the tensor cores work on one row tile while the
// other's exponentials are formed, and K and V serve 256 rows per load.
//
// Order of the matrix instructions: ... O_0 += P_0 V_j, S_0 = Q_0 K_j+1, O_1 += P_1 V_j, S_1 = Q_1 K_j+1 ...
// They complete in issue order, so S_t of the next tile may overwrite P_t, and a softmax thread that
// has seen S_t(j+1) also knows that O_t(j) is complete.  The products with the first half of P begin while the
// second half's exponentials are formed (1454 -> 1496 TFLOP/s at 4096 rows, 8192 states, 16 heads of 128, 4 graphs).
//
// Bound: the chain S - exponentials - O of a row tile.  Per tile of 128 x 128 the products take some 1020 clocks at head
// dimension 128 (about 580 at 64) and the exponentials 512 (32 a clock and SM), and with two row tiles an SM one's
// exponentials overlap the other's products, less the waits between the roles: 1760 clocks a tile at 128, 1490 at 64
// (405 and 340 us for 16 heads, 4 x 4096 rows and states).  Tried and slower: steps of 64 states with two or three S
// (848 -> 1050 us), two warpgroups a row tile.  P is rounded to 16 bits for its product with V, which takes 16-bit operands;
// its sum l is of the unrounded values.  Single tokens over long encodings
// are bound by memory: 8 x 16384 states, 32/8 heads of 128: 101 us, 5290 GB/s; ragged lengths to 16384 72 us, 3780 GB/s.
#include "attn_mma.h"

namespace uvu {
namespace {

constexpr int kMaskRing = 8;  // state masks in flight: more than half the stages, plus two

// Shared memory of the forward: NT row tiles of Q, the ring of K and V tiles, masks, barriers.
template <int NT>
struct FwdLayout {
    int panels, stages;
    int masks_held;  // biases of state tiles in flight: kMaskRing, or 1 without a mask (the last tile's)
    __host__ __device__ int tile() const { return panels * kPanelBytes; }
    __host__ __device__ int ring() const { return NT * tile(); }
    __host__ __device__ int masks() const { return ring() + stages * tile(); }
    __host__ __device__ int bars() const { return masks() + masks_held * kRows * 4; }
    __host__ __device__ int total() const { return bars() + 288 + 1024; }  // barriers, alignment slack
};

// Adds a row of O to what a long walk holds of it (null: a lane without a row), held so far at another reference by the factor f.
static __device__ __noinline__ void hold_row(uint32_t o_at, int D, float* held, float f, bool first) {
    for (int d = 0; d < D; d += 16) {
        float o[16];
        __syncwarp();
        tmem_ld16(o_at + d, o);
        tmem_wait_ld(o);
        if (!held) continue;
        if (D % 4 == 0) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                if (d + i < D) {
                    float4* at = reinterpret_cast<float4*>(held + d + i);
                    const float4 h = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *at;
                    *at = make_float4(fmaf(h.x, f, o[i]), fmaf(h.y, f, o[i + 1]), fmaf(h.z, f, o[i + 2]), fmaf(h.w, f, o[i + 3]));
                }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (d + i < D) held[d + i] = fmaf(first ? 0.f : held[d + i], f, o[i]);
        }
    }
}

// HELD: long walks, whose sums leave tensor memory every kHold tiles (as a branch of the one kernel it cost single tokens over long
// encodings 2%).
template <typename T, int NT, int LG, bool ALIGNED, bool HELD>
__global__ void __launch_bounds__((4 * NT + 1 + kLoadWarps) * 32, NT == 1 && LG < 4 ? 2 : 1) attn_fwd_mma(AttnArgs a, FwdLayout<NT> L) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ int s_dead, s_kept;  // s_kept: a mask has kept one of the piece's states
    __shared__ uint32_t s_tmem;
    const AttnTile tl = attn_tile<kRows * NT>(a.q_off, a.k_off, a.graphs, a.group, blockIdx.x);
    if (tl.graph < 0) return;
    const int h = blockIdx.y, split = blockIdx.z;
    const int64_t q0 = tl.first, k0 = tl.other;
    const Piece kr = piece_of(tl.n, split, a.splits);
    const int n_tiles = uniform(int((kr.hi - kr.lo + kRows - 1) / kRows));
    const int n_rows = uniform(int(min(tl.rows - tl.row0, int64_t(kRows * NT))));
    const int nt = NT == 2 && n_rows > kRows ? 2 : 1;  // row tiles in use
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = uniform(smem_u32(smem));
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int d16 = (a.D + 15) / 16;
    const uint32_t q_full = sb + L.bars(), s_full = q_full + 8, p_half = s_full + 16, p_full = p_half + 16, o_full = p_full + 16, full = o_full + 16,
                   empty = full + 8 * L.stages, m_full = empty + 8 * L.stages, fin = m_full + 8 * kMaskRing;
    const uint32_t o_cols = uint32_t(64 * L.panels);
    const uint32_t tmem_cols = NT == 2 ? 512 : 256;
    if (threadIdx.x == 0) {
        s_dead = s_kept = 0;
        bar_init(q_full, kLoadWarps * 32);
        for (int t = 0; t < 2; ++t) {
            bar_init(s_full + 8 * t, 1);
            bar_init(p_half + 8 * t, 4);
            bar_init(p_full + 8 * t, 4);
            bar_init(o_full + 8 * t, 1);
        }
        for (int s = 0; s < L.stages; ++s) {
            bar_init(full + 8 * s, kLoadWarps * 32);
            bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < kMaskRing; ++s) bar_init(m_full + 8 * s, kLoadThreads);
        bar_init(fin, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4 * NT) tmem_alloc(smem_u32(&s_tmem), tmem_cols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(&s_tmem));
    volatile int* dead = &s_dead;
    unsigned* status = &attn_status_word;
    float* biases = reinterpret_cast<float*>(smem + L.masks());
    // the bias of tile j: every tile's with a mask, else the last one's where it is not full
    const bool tail = (kr.hi - kr.lo) % kRows != 0;
    auto masked = [&](int j) { return a.keep || (tail && j == n_tiles - 1); };
    auto slot = [&](int j) { return a.keep ? j % kMaskRing : 0; };
    // O begins anew at these tiles
    constexpr int kHold = attn_hold_tiles(__is_same(T, __half));
    const bool held = HELD && n_tiles > kHold;
    auto fresh = [&](int j) { return j == 0 || (HELD && j % kHold == 0); };

    if (warp < 4 * NT) {
        // ------------------------------------------------------------------------ softmax
        const int t = warp >> 2, quad = warp & 3;
        const int row = t * kRows + quad * 32 + lane;
        const bool work = t * kRows + quad * 32 < n_rows;  // the warp has rows
        const uint32_t lanes = uint32_t(quad * 32) << 16;
        const uint32_t s_at = tmem + uint32_t(t * kRows) + lanes, o_at = tmem + uint32_t(NT * kRows) + uint32_t(t) * o_cols + lanes;
        const float c = a.scale_log2;
        float m = -INFINITY, l = 0.f;  // reference maximum in units of c S, and the sum of P
        float m_held = -INFINITY;      // the reference of what is held in memory
        auto held_row = [&]() {
            const int64_t p = tl.row0 + row, rh = (int64_t(split) * a.nq + q0 + p / a.group) * a.Hq + int64_t(h) * a.group + p % a.group;
            return a.part_o + rh * a.D;
        };
        auto held_factor = [&]() { return m_held == m ? 1.f : exp2_approx(m_held - m); };
        bool ok = true;
        if (t < nt) {
            // a block with all of an SM's registers holds its row of S; the others read it twice
            constexpr bool kKeep = NT == 2 || LG == 4;
            for (int j = 0; j < n_tiles; ++j) {
                const bool biased = masked(j);
                const float* bias = biases + slot(j) * kRows;
                if (biased) {
                    ok = warp_wait(m_full + 8 * slot(j), a.keep ? (j / kMaskRing) & 1 : 0, dead, status);
                    if (!ok) break;
                }
                ok = warp_wait(s_full + 8 * t, j & 1, dead, status);
                if (!ok) break;
                fence_after();
                if (work) {
                    if (HELD && j > 0 && fresh(j)) {  // O of the tile before is complete
                        hold_row(o_at, a.D, row < n_rows ? held_row() : nullptr, held_factor(), j == kHold);
                        m_held = m;
                    }
                    float x[kKeep ? 4 : 2][32];
                    float top = -INFINITY;
                    if constexpr (kKeep) {
#pragma unroll
                        for (int b = 0; b < 4; ++b) tmem_ld32(s_at + 32 * b, x[b]);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            tmem_wait_ld(x[b]);
                            if (biased) add_bias(x[b], bias + 32 * b);
                        }
                        const float t0 = fmaxf(row_max(x[0]), row_max(x[1])), t1 = fmaxf(row_max(x[2]), row_max(x[3]));
                        top = fmaxf(t0, t1);
                    } else {
                        tmem_ld32(s_at, x[0]);
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            float(&v)[32] = x[b & 1];
                            tmem_wait_ld(v);
                            tmem_ld32(s_at + 32 * ((b + 1) & 3), x[(b + 1) & 1]);
                            if (biased) add_bias(v, bias + 32 * b);
                            top = fmaxf(top, row_max(v));
                        }
                    }
                    top *= c;
                    const bool move = top > m + 8.f;
                    if (__any_sync(0xffffffffu, move)) {
                        const float to = move ? top : m;
                        if (j > 0) {
                            const float f = move ? exp2_approx(m - to) : 1.f;
                            l *= f;
                            for (int d = 0; d < (fresh(j) ? 0 : d16); ++d) {
                                float o[16];
                                tmem_ld16(o_at + 16 * d, o);
                                tmem_wait_ld(o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= f;
                                tmem_st16(o_at + 16 * d, o);
                            }
                        }
                        m = to;
                    }
                    const float base = m == -INFINITY ? 0.f : m;
                    const F2 c2(c, c), minus(-base, -base);
                    F2 sum[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        float(&v)[32] = x[kKeep ? b : b & 1];
                        if constexpr (!kKeep) {
                            tmem_wait_ld(v);
                            if (b < 3) tmem_ld32(s_at + 32 * (b + 1), x[(b + 1) & 1]);
                            if (biased) add_bias(v, bias + 32 * b);
                        }
                        exp_row(v, c2, minus, sum);
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) p[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
                        tmem_st16(s_at + 16 * b, p);
                        if (b == 1) {
                            tmem_wait_st();
                            fence_before();
                            __syncwarp();
                            if (lane == 0) bar_arrive(p_half + 8 * t);
                        }
                    }
                    const float2 s2 = (sum[0] + sum[1]).both();
                    l += s2.x + s2.y;
                    tmem_wait_st();
                }
                fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (!work) bar_arrive(p_half + 8 * t);
                    bar_arrive(p_full + 8 * t);
                }
            }
            if (ok && n_tiles > 0) {
                ok = warp_wait(o_full + 8 * t, 0, dead, status);
                fence_after();
            }
            if (ok && work) {
                const bool valid = row < n_rows;
                if (a.keep && !*static_cast<volatile int*>(&s_kept)) l = 0.f;  // nothing to attend to, whatever q holds
                const float inv = l == 0.f ? 0.f : 1.f / l, f = held ? held_factor() : 0.f;
                const int64_t p = tl.row0 + row;
                const int64_t r = q0 + p / a.group, head = int64_t(h) * a.group + p % a.group;
                const int64_t rh = (int64_t(split) * a.nq + r) * a.Hq + head;
                if (valid) (a.splits > 1 ? a.part_lse[rh] : a.lse[r * a.Hq + head]) = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                T* out = static_cast<T*>(a.out) + r * a.o_row + head * a.o_head;
                const bool vec = ((reinterpret_cast<uintptr_t>(a.out) | uintptr_t(a.o_row * 2) | uintptr_t(a.o_head * 2)) & 15u) == 0;
                for (int d = 0; d < d16; ++d) {
                    float o[16];
                    __syncwarp();
                    if (n_tiles > 0) {
                        tmem_ld16(o_at + 16 * d, o);
                        tmem_wait_ld(o);
                    }
                    if (held && valid) {
                        const float* from = a.part_o + rh * a.D + 16 * d;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (16 * d + i < a.D) o[i] = fmaf(from[i], f, o[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = l == 0.f ? 0.f : o[i] * inv;
                    if (!valid) {
                        // a row past the end: read with its warp, stored nowhere
                    } else if (a.splits > 1) {
                        float* po = a.part_o + rh * a.D + 16 * d;
                        if (a.D % 4 == 0) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (16 * d + 4 * i < a.D)
                                    *reinterpret_cast<float4*>(po + 4 * i) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (16 * d + i < a.D) po[i] = o[i];
                        }
                    } else if (vec && a.D % 8 == 0) {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if (16 * d + 8 * i < a.D)
                                *reinterpret_cast<uint4*>(out + 16 * d + 8 * i) =
                                    make_uint4(pack2<T>(o[8 * i], o[8 * i + 1]), pack2<T>(o[8 * i + 2], o[8 * i + 3]),
                                               pack2<T>(o[8 * i + 4], o[8 * i + 5]), pack2<T>(o[8 * i + 6], o[8 * i + 7]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (16 * d + i < a.D) out[16 * d + i] = narrow<T>(o[i]);
                    }
                }
            }
        }
    } else if (warp == 4 * NT) {
        // ----------------------------------------------------------------- matrix instructions
        {
            const uint32_t lead = elect_lane();
            const uint32_t id_s = mma_desc<T>(kRows, false), id_o = mma_desc<T>(16 * d16, true);
            Ring ring(L.stages);
            auto wait_stage = [&]() { return warp_wait(full + 8 * ring.at, ring.parity, dead, status); };
            auto stage = [&]() { return sb + uint32_t(L.ring() + ring.at * L.tile()); };
            auto scores = [&](int t, uint32_t k) {
                const uint32_t q = sb + uint32_t(t * L.tile());
#pragma unroll
                for (int s = 0; s < 1 << (LG - 1); ++s)  // all of them, or fewer off the class's largest head dimension
                    if (s < d16) mma_ss(lead, tmem + uint32_t(t * kRows), desc_cols(q, s), desc_cols(k, s), id_s, s > 0);
                mma_commit(lead, s_full + 8 * t);
            };
            bool ok = n_tiles > 0 && warp_wait(q_full, 0, dead, status) && wait_stage();
            if (ok) {
                fence_async();
                for (int t = 0; t < nt; ++t) scores(t, stage());
                mma_commit(lead, empty + 8 * 0);
                ring.next();
            }
            for (int j = 0; j < n_tiles && ok; ++j) {
                ok = wait_stage();
                fence_async();
                const bool more = !fresh(j);
                const int v_at = ring.at;
                const uint32_t v = stage();
                ring.next();
                const uint32_t k = stage();
                for (int t = 0; t < nt && ok; ++t) {
                    const uint32_t o = tmem + uint32_t(NT * kRows) + uint32_t(t) * o_cols;
#pragma unroll
                    for (int half = 0; half < 2 && ok; ++half) {
                        ok = warp_wait((half ? p_full : p_half) + 8 * t, j & 1, dead, status);
                        if (!ok) break;
                        fence_after();
#pragma unroll
                        for (int s = 4 * half; s < 4 * half + 4; ++s)
                            mma_ts(lead, o, tmem + uint32_t(t * kRows + 8 * s), desc_rows(v, s), id_o, more || s > 0);
                    }
                    if (!ok) break;
                    if (j + 1 < n_tiles) {
                        if (t == 0) {
                            ok = wait_stage();
                            if (!ok) break;
                            fence_async();
                        }
                        scores(t, k);
                    } else {
                        mma_commit(lead, o_full + 8 * t);
                    }
                }
                if (!ok) break;
                mma_commit(lead, empty + 8 * v_at);
                if (j + 1 < n_tiles) mma_commit(lead, empty + 8 * ring.at);
                ring.next();
            }
            // every instruction issued has finished before the tensor memory and the stages go
            mma_commit(lead, fin);
            bar_wait_last(fin, 0, status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------------- loaders
        const int map_t = threadIdx.x - (4 * NT + 1) * 32;
        const LoadMap<LG> map(map_t, a.D);
        if (n_tiles > 0) {
            // every loader thread arrives: when its copies have landed, or at once after its own stores
            auto arrive = [&](uint32_t bar) { ALIGNED ? copy_arrive(bar) : bar_arrive(bar); };
            const char* Q = reinterpret_cast<const char*>(static_cast<const T*>(a.q) + q0 * a.q_row + int64_t(h) * a.group * a.q_head);
            for (int i = 0; i < nt; ++i)
                load_packed<ALIGNED, false>(sb + uint32_t(i * L.tile()), Q, a.q_row * 2, a.q_head * 2, a.group, tl.row0 + i * kRows,
                                         n_rows - i * kRows, map);
            arrive(q_full);
            const char* K = reinterpret_cast<const char*>(static_cast<const T*>(a.k) + (k0 + kr.lo) * a.k_row + h * a.k_head) + map.chunk * 16;
            const char* V = reinterpret_cast<const char*>(static_cast<const T*>(a.v) + (k0 + kr.lo) * a.v_row + h * a.v_head) + map.chunk * 16;
            StateMask<> mask(a.keep ? a.keep + k0 : nullptr, kr.lo, kr.hi);
            Ring ring(L.stages);
            auto load = [&](const char* src, int64_t stride) {
                if (ring.uses >= L.stages && !warp_wait(empty + 8 * ring.at, ring.parity ^ 1, dead, status)) return false;
                const uint32_t dst = sb + uint32_t(L.ring() + ring.at * L.tile());
                load_states<ALIGNED>(dst, src, stride, map, mask);
                arrive(full + 8 * ring.at);
                ring.next();
                return true;
            };
            for (int j = 0; j < n_tiles; ++j) {
                mask.next();
                if (!load(K, a.k_row * 2)) break;
                // the softmax warps read the tile's bias before its V stage is released, and K's stage comes half a ring
                // later: kMaskRing biases cannot be overtaken
                if (masked(j)) {
                    if (map_t == 0 && mask.any()) s_kept = 1;
                    write_bias(biases + slot(j) * kRows, mask, map_t);
                    bar_arrive(m_full + 8 * slot(j));
                }
                if (!load(V, a.v_row * 2)) break;
                K += kRows * a.k_row * 2;
                V += kRows * a.v_row * 2;
            }
            copy_wait_all();
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 4 * NT) {
        fence_after();
        tmem_free(tmem, tmem_cols);
    }
}

template <typename T, int NT>
cudaError_t fwd(const AttnArgs& a, int64_t row_tiles, cudaStream_t st) {
    FwdLayout<NT> L;
    L.panels = a.D > 64 ? 2 : 1;
    // one panel: 96 KB, two CTAs per SM (NT = 1), or 160 KB; two panels: 224 KB, less
    // a stage where the masks need the room
    L.masks_held = a.keep ? kMaskRing : 1;
    L.stages = NT == 1 ? (L.panels == 1 || a.keep ? 5 : 6) : (L.panels == 1 ? 8 : a.keep ? 4 : 5);
    const uintptr_t any = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                          uintptr_t(a.q_row | a.q_head | a.k_row | a.k_head | a.v_row | a.v_head) * 2;
    return by_chunks(a.D, (any & 15u) == 0, [&](auto lg, auto aligned) {
        constexpr int LG = decltype(lg)::value;
        constexpr bool ALIGNED = decltype(aligned)::value;
        auto k = a.hold ? attn_fwd_mma<T, NT, LG, ALIGNED, true> : attn_fwd_mma<T, NT, LG, ALIGNED, false>;
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L.total());
        if (e != cudaSuccess) return e;
        k<<<dim3(unsigned(row_tiles), unsigned(a.Hkv), unsigned(a.splits)), (4 * NT + 1 + kLoadWarps) * 32, L.total(), st>>>(a, L);
        return cudaGetLastError();
    });
}

}  // namespace

cudaError_t launch_attn_fwd_mma(uvu_dtype dtype, const AttnArgs& a, int nt, int64_t row_tiles, cudaStream_t st) {
    if (dtype == UVU_BF16) return nt == 2 ? fwd<__nv_bfloat16, 2>(a, row_tiles, st) : fwd<__nv_bfloat16, 1>(a, row_tiles, st);
    return nt == 2 ? fwd<__half, 2>(a, row_tiles, st) : fwd<__half, 1>(a, row_tiles, st);
}

cudaError_t attn_fwd_mma_status(unsigned* word, bool reset) { return read_status(word, reset); }

}  // namespace uvu
