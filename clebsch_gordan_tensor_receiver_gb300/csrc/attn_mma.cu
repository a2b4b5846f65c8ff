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
// instructions, four warps that load.  With NT = 2 the tensor cores work on one row tile while the
// other's exponentials are formed, and K and V serve 256 rows per load.  The loaders use 16-byte
// cp.async with zero fill instead of tensor maps: a masked or absent state is zeros in shared memory,
// whatever memory holds there (0 * NaN would reach O), and any row and head strides work; operands off
// the 16-byte grid go through registers.  A stage is handed on when its copies have landed, kLag
// stages after they were issued.
//
// Order of the matrix instructions: ... O_0 += P_0 V_j, S_0 = Q_0 K_j+1, O_1 += P_1 V_j, S_1 = Q_1 K_j+1 ...
// They complete in issue order, so S_t of the next tile may overwrite P_t, and a softmax thread that
// has seen S_t(j+1) also knows that O_t(j) is complete.
//
// Every wait is bounded (two seconds); on expiry the roles leave their loops, the issuer waits for its
// instructions, the loaders for their copies, and the CTA frees its tensor memory and returns with the
// status word set.
#include <algorithm>
#include <cstdint>

#include "attn.h"
#include "elem.h"
#include "tensor_core.h"

namespace uvu {

__device__ unsigned int attn_status_word;

namespace {

using namespace tc;

constexpr int kRows = 128;      // rows of a row tile, states of a state tile
constexpr int kMaskRing = 8;    // state masks in flight: more than half the stages, plus two
constexpr int kLoadWarps = 2;
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kLoadThreads = kLoadWarps * 32;

// How the loader threads share a tile of 128 rows: thread t takes 16-byte chunk t % 2^LG of the rows
// t / 2^LG, + kStep, ...  2^LG is the power of two that holds the row's chunks.
template <int LG>
struct LoadMap {
    static constexpr int kStep = kLoadThreads >> LG, kIters = kRows / kStep;
    int row, chunk;
    uint32_t bytes;  // of the chunk that exist: the others are zeros
    bool on;         // the chunk is read by the matrix instructions
    __device__ __forceinline__ LoadMap(int t, int D)
        : row(t >> LG), chunk(t & ((1 << LG) - 1)), bytes(uint32_t(min(max(D - 8 * chunk, 0), 8)) * 2), on(chunk < 2 * ((D + 15) / 16)) {}
};

// One 16-byte chunk (of which `bytes` exist) into shared memory.
template <bool ALIGNED>
__device__ __forceinline__ void load_chunk(uint32_t to, const char* src, uint32_t bytes) {
    if constexpr (ALIGNED) {
        copy16(to, src, bytes);
    } else {
        uint32_t w[4] = {0, 0, 0, 0};
        const uint16_t* p = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (2 * i < bytes) w[i >> 1] |= uint32_t(p[i]) << (16 * (i & 1));
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    }
}

// 128 rows with a constant stride, `src` the first (its chunk included); rows that `use` refuses are
// zeros.  ALL: every row is used.
template <int LG, bool ALIGNED, bool ALL, typename Use>
__device__ __forceinline__ void load_strided(uint32_t dst, const char* src, int64_t stride, const LoadMap<LG>& m, Use use) {
    using M = LoadMap<LG>;
    if (!m.on) return;
    // rows kStep apart share their swizzle when kStep is a multiple of 8; at 4 it alternates
    const uint32_t even = dst + tile_offset(m.row, m.chunk), odd = dst + tile_offset(m.row + M::kStep, m.chunk) - uint32_t(M::kStep * 128);
    const char* p = src + m.row * stride;
#pragma unroll 8
    for (int i = 0; i < M::kIters; ++i) {
        load_chunk<ALIGNED>((i & 1 ? odd : even) + uint32_t(i * M::kStep * 128), p, ALL || use(m.row + i * M::kStep) ? m.bytes : 0);
        p += M::kStep * stride;
    }
}

// Packed rows r0 .. r0 + 128 of a kv head's queries: row r is query r / group, head r % group.
template <int LG, bool ALIGNED>
__device__ __forceinline__ void load_packed(uint32_t dst, const char* base, int64_t row, int64_t head, int group, int64_t r0, int rows,
                                            const LoadMap<LG>& m) {
    using M = LoadMap<LG>;
    if (group == 1) {
        auto use = [&](int r) { return r < rows; };
        if (rows >= kRows)
            load_strided<LG, ALIGNED, true>(dst, base + r0 * row + m.chunk * 16, row, m, use);
        else
            load_strided<LG, ALIGNED, false>(dst, base + r0 * row + m.chunk * 16, row, m, use);
        return;
    }
    if (!m.on) return;
    // query and head of the thread's first row; later rows step by kStep without a division
    const uint32_t g = uint32_t(group), dq = uint32_t(M::kStep) / g, dj = uint32_t(M::kStep) - dq * g;
    const int64_t q0 = (r0 + m.row) / group;
    uint32_t j = uint32_t(r0 + m.row - q0 * group);
    const char* p = base + q0 * row + int64_t(j) * head + m.chunk * 16;
    const int64_t step = dq * row + int64_t(dj) * head, wrap = row - int64_t(g) * head;
#pragma unroll 4
    for (int i = 0; i < M::kIters; ++i) {
        const int r = m.row + i * M::kStep;
        load_chunk<ALIGNED>(dst + tile_offset(r, m.chunk), p, r < rows ? m.bytes : 0);
        p += step;
        j += dj;
        if (j >= g) {
            j -= g;
            p += wrap;
        }
    }
}

__device__ __forceinline__ uint32_t tail_word(int64_t left, int w) {  // bits of the states that exist
    const int64_t n = left - 32 * w;
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << uint32_t(n)) - 1u;
}

// Which of a tile's 128 states take part, as four words in every lane of a loader warp.  The mask
// bytes of the next tile are fetched a tile ahead.
struct StateMask {
    const uint8_t* keep;  // of the graph, or null
    int64_t at, hi;       // first state of the coming tile, end
    uint32_t word[4], ahead;
    __device__ __forceinline__ StateMask(const uint8_t* k, int64_t lo, int64_t end) : keep(k), at(lo), hi(end), ahead(0) { fetch(); }
    __device__ __forceinline__ void fetch() {
        if (!keep) return;
        ahead = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int64_t s = at + 32 * w + (threadIdx.x & 31);
            if (s < hi && keep[s]) ahead |= 1u << w;
        }
    }
    __device__ __forceinline__ void next() {
#pragma unroll
        for (int w = 0; w < 4; ++w) word[w] = keep ? __ballot_sync(0xffffffffu, (ahead >> w) & 1) : tail_word(hi - at, w);
        at += kRows;
        fetch();
    }
    __device__ __forceinline__ bool all() const { return (word[0] & word[1] & word[2] & word[3]) == 0xffffffffu; }
    __device__ __forceinline__ bool has(int r) const {
        const uint32_t w = r < 64 ? (r < 32 ? word[0] : word[1]) : (r < 96 ? word[2] : word[3]);
        return (w >> (r & 31)) & 1;
    }
};

struct Piece {
    int64_t lo, hi;
};
__device__ __forceinline__ Piece piece_of(int64_t n, int s, int splits) {
    const int64_t tiles = (n + kRows - 1) / kRows, per = (tiles + splits - 1) / splits;
    return {min(n, s * per * kRows), min(n, (s + 1) * per * kRows)};
}

// Shared memory of the forward: NT row tiles of Q, the ring of K and V tiles, masks, barriers.
template <int NT>
struct FwdLayout {
    int panels, stages;
    __host__ __device__ int tile() const { return panels * kPanelBytes; }
    __host__ __device__ int ring() const { return NT * tile(); }
    __host__ __device__ int masks() const { return ring() + stages * tile(); }
    __host__ __device__ int bars() const { return masks() + kMaskRing * 16; }
    __host__ __device__ int total() const { return bars() + 256 + 1024; }  // + alignment slack
};

template <typename T, int NT, int LG, bool ALIGNED>
__global__ void __launch_bounds__((4 * NT + 1 + kLoadWarps) * 32, NT == 1 ? 2 : 1) attn_fwd_mma(AttnArgs a, FwdLayout<NT> L) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ int s_dead;
    __shared__ uint32_t s_tmem;
    const AttnTile tl = attn_tile(a.q_off, a.graphs, a.group, kRows * NT, blockIdx.x);
    if (tl.graph < 0) return;
    const int h = blockIdx.y, split = blockIdx.z;
    const int64_t q0 = a.q_off[tl.graph], k0 = a.k_off[tl.graph];
    const Piece kr = piece_of(a.k_off[tl.graph + 1] - k0, split, a.splits);
    const int n_tiles = int((kr.hi - kr.lo + kRows - 1) / kRows);
    const int n_rows = int(min(tl.rows - tl.row0, int64_t(kRows * NT)));
    const int nt = NT == 2 && n_rows > kRows ? 2 : 1;  // row tiles in use
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int d16 = (a.D + 15) / 16;
    const uint32_t q_full = sb + L.bars(), s_full = q_full + 8, p_full = s_full + 16, o_full = p_full + 16, full = o_full + 16,
                   empty = full + 8 * L.stages, m_full = empty + 8 * L.stages, fin = m_full + 8 * kMaskRing;
    const uint32_t o_cols = uint32_t(64 * L.panels);
    const uint32_t tmem_cols = NT == 2 ? 512 : 256;
    if (threadIdx.x == 0) {
        s_dead = 0;
        bar_init(q_full, kLoadWarps * 32);
        for (int t = 0; t < 2; ++t) {
            bar_init(s_full + 8 * t, 1);
            bar_init(p_full + 8 * t, 4);
            bar_init(o_full + 8 * t, 1);
        }
        for (int s = 0; s < L.stages; ++s) {
            bar_init(full + 8 * s, kLoadWarps * 32);
            bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < kMaskRing; ++s) bar_init(m_full + 8 * s, 1);
        bar_init(fin, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 4 * NT) tmem_alloc(smem_u32(&s_tmem), tmem_cols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
    volatile int* dead = &s_dead;
    unsigned* status = &attn_status_word;
    const uint32_t* masks = reinterpret_cast<const uint32_t*>(smem + L.masks());

    if (warp < 4 * NT) {
        // ------------------------------------------------------------------------ softmax
        const int t = warp >> 2, quad = warp & 3;
        const int row = t * kRows + quad * 32 + lane;
        const bool work = t * kRows + quad * 32 < n_rows;  // the warp has rows
        const uint32_t lanes = uint32_t(quad * 32) << 16;
        const uint32_t s_at = tmem + uint32_t(t * kRows) + lanes, o_at = tmem + uint32_t(NT * kRows) + uint32_t(t) * o_cols + lanes;
        const float c = a.scale_log2;
        float m = -INFINITY, l = 0.f;  // reference maximum in units of c S, and the sum of P
        bool ok = true;
        if (t < nt) {
            for (int j = 0; j < n_tiles; ++j) {
                uint32_t word[4];
                if (a.keep) {
                    ok = __all_sync(0xffffffffu, bar_wait(m_full + 8 * (j % kMaskRing), (j / kMaskRing) & 1, dead, status));
                    if (!ok) break;
#pragma unroll
                    for (int w = 0; w < 4; ++w) word[w] = masks[(j % kMaskRing) * 4 + w];
                } else {
#pragma unroll
                    for (int w = 0; w < 4; ++w) word[w] = tail_word(kr.hi - kr.lo - int64_t(j) * kRows, w);
                }
                ok = __all_sync(0xffffffffu, bar_wait(s_full + 8 * t, j & 1, dead, status));
                if (!ok) break;
                fence_after();
                if (work) {
                    float x[2][32];
                    float top = -INFINITY;
                    tmem_ld32(s_at, x[0]);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        float(&v)[32] = x[b & 1];
                        tmem_wait_ld(v);
                        tmem_ld32(s_at + 32 * ((b + 1) & 3), x[(b + 1) & 1]);
                        if (word[b] == 0xffffffffu) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) top = fmaxf(top, v[i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if ((word[b] >> i) & 1) top = fmaxf(top, v[i]);
                        }
                    }
                    top *= c;
                    const bool move = top > m + 8.f;
                    if (__any_sync(0xffffffffu, move)) {
                        const float to = move ? top : m;
                        if (j > 0) {
                            const float f = move ? exp2_approx(m - to) : 1.f;
                            l *= f;
                            for (int d = 0; d < d16; ++d) {
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
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        float(&v)[32] = x[b & 1];
                        tmem_wait_ld(v);
                        if (b < 3) tmem_ld32(s_at + 32 * (b + 1), x[(b + 1) & 1]);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = exp2_approx(fmaf(v[i], c, -base));
                        if (word[b] != 0xffffffffu) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((word[b] >> i) & 1)) v[i] = 0.f;
                        }
                        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[i & 3] += v[i];
                        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) p[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
                        tmem_st16(s_at + 16 * b, p);
                    }
                    tmem_wait_st();
                }
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(p_full + 8 * t);
            }
            if (ok && n_tiles > 0) {
                ok = __all_sync(0xffffffffu, bar_wait(o_full + 8 * t, 0, dead, status));
                fence_after();
            }
            if (ok && work) {
                const bool valid = row < n_rows;
                const float inv = l == 0.f ? 0.f : 1.f / l;
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
        if (lane == 0) {
            const uint32_t id_s = mma_desc<T>(kRows, false), id_o = mma_desc<T>(16 * d16, true);
            auto stage = [&](int i) { return sb + uint32_t(L.ring() + (i % L.stages) * L.tile()); };
            auto wait_stage = [&](int i) { return bar_wait(full + 8 * (i % L.stages), (i / L.stages) & 1, dead, status); };
            auto scores = [&](int t, int j) {
                const uint32_t q = sb + uint32_t(t * L.tile()), k = stage(2 * j);
                for (int s = 0; s < d16; ++s) mma_ss(tmem + uint32_t(t * kRows), desc_cols(q, s), desc_cols(k, s), id_s, s > 0);
                mma_commit(s_full + 8 * t);
            };
            bool ok = n_tiles > 0 && bar_wait(q_full, 0, dead, status) && wait_stage(0);
            if (ok) {
                fence_async();
                for (int t = 0; t < nt; ++t) scores(t, 0);
                mma_commit(empty + 8 * 0);
            }
            for (int j = 0; j < n_tiles && ok; ++j) {
                ok = wait_stage(2 * j + 1);
                fence_async();
                for (int t = 0; t < nt && ok; ++t) {
                    ok = bar_wait(p_full + 8 * t, j & 1, dead, status);
                    if (!ok) break;
                    fence_after();
                    const uint32_t o = tmem + uint32_t(NT * kRows) + uint32_t(t) * o_cols, v = stage(2 * j + 1);
#pragma unroll
                    for (int s = 0; s < kRows / 16; ++s)
                        mma_ts(o, tmem + uint32_t(t * kRows + 8 * s), desc_rows(v, s), id_o, j > 0 || s > 0);
                    if (j + 1 < n_tiles) {
                        if (t == 0) {
                            ok = wait_stage(2 * j + 2);
                            if (!ok) break;
                            fence_async();
                        }
                        scores(t, j + 1);
                    } else {
                        mma_commit(o_full + 8 * t);
                    }
                }
                if (!ok) break;
                mma_commit(empty + 8 * ((2 * j + 1) % L.stages));
                if (j + 1 < n_tiles) mma_commit(empty + 8 * ((2 * j + 2) % L.stages));
            }
            // every instruction issued has finished before the tensor memory and the stages go
            mma_commit(fin);
            bar_wait_last(fin, 0, status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------------- loaders
        const LoadMap<LG> map(threadIdx.x - (4 * NT + 1) * 32, a.D);
        if (n_tiles > 0) {
            // every loader thread arrives: when its copies have landed, or at once after its own stores
            auto arrive = [&](uint32_t bar) { ALIGNED ? copy_arrive(bar) : bar_arrive(bar); };
            const char* Q = reinterpret_cast<const char*>(static_cast<const T*>(a.q) + q0 * a.q_row + int64_t(h) * a.group * a.q_head);
            for (int i = 0; i < nt; ++i)
                load_packed<LG, ALIGNED>(sb + uint32_t(i * L.tile()), Q, a.q_row * 2, a.q_head * 2, a.group, tl.row0 + i * kRows,
                                         n_rows - i * kRows, map);
            arrive(q_full);
            const char* K = reinterpret_cast<const char*>(static_cast<const T*>(a.k) + (k0 + kr.lo) * a.k_row + h * a.k_head) + map.chunk * 16;
            const char* V = reinterpret_cast<const char*>(static_cast<const T*>(a.v) + (k0 + kr.lo) * a.v_row + h * a.v_head) + map.chunk * 16;
            StateMask mask(a.keep ? a.keep + k0 : nullptr, kr.lo, kr.hi);
            auto load = [&](int i, const char* src, int64_t stride) {
                if (i >= L.stages &&
                    !__all_sync(0xffffffffu, bar_wait(empty + 8 * (i % L.stages), (i / L.stages - 1) & 1, dead, status)))
                    return false;
                const uint32_t dst = sb + uint32_t(L.ring() + (i % L.stages) * L.tile());
                auto use = [&](int r) { return mask.has(r); };
                if (mask.all())
                    load_strided<LG, ALIGNED, true>(dst, src, stride, map, use);
                else
                    load_strided<LG, ALIGNED, false>(dst, src, stride, map, use);
                arrive(full + 8 * (i % L.stages));
                return true;
            };
            for (int j = 0; j < n_tiles; ++j) {
                mask.next();
                if (!load(2 * j, K, a.k_row * 2)) break;
                // the softmax warps read the tile's mask before its V stage is released, and K's stage comes half a ring
                // later: kMaskRing masks cannot be overtaken
                if (a.keep && warp == 4 * NT + 1 && lane == 0) {
                    *reinterpret_cast<uint4*>(smem + L.masks() + (j % kMaskRing) * 16) =
                        make_uint4(mask.word[0], mask.word[1], mask.word[2], mask.word[3]);
                    bar_arrive(m_full + 8 * (j % kMaskRing));
                }
                if (!load(2 * j + 1, V, a.v_row * 2)) break;
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

// ------------------------------------------------------------------------------------ backward

// KV false: dq of a tile of 128 packed rows, walking the states; KV true: dk and dv of a tile of 128
// states, walking the packed rows of all heads that share them (so a shared head's gradient needs no
// second sum).  R1, R2: the tile's own operands, resident; X1, X2: the walked ones, in the ring.
//              R1  R2  X1  X2      S = R1 X1^T,  dP = R2 X2^T,  P = exp2(c S - lse),  dS = P (dP - delta)
//     dq       Q   dO  K   V       dq += dS X1
//     dk, dv   K   V   Q   dO      dk += dS X1,  dv += P X2      (S and dP transposed: lanes are states)
// Two sweeps instead of one cost S and dP twice (seven products instead of five), but every sum stays
// in one CTA's tensor memory: no atomics, and results that do not depend on timing.
//
// Tensor memory: S, dP (128 columns each), then the sums.  P and dS are written as 16-bit values over
// the part of S and dP that the same thread has read.  Two warpgroups share a tile: warpgroup w takes
// columns 64 w .. + 63 of each lane's row.  Order of the matrix instructions:
//     S(0) dP(0) | dv += P(0) X2, S(1), dk += dS(0) X1, dP(1) | ...
// so the tensor cores form dv(j) and S(j+1) while the threads turn dP(j) into dS(j), and dk(j) and
// dP(j+1) while they turn S(j+1) into P(j+1).
//
// f16 keeps 2^8 P (undone in the epilogue and in dS): P of long rows would fall below the type's
// smallest normal value, 2^-14.  bf16 has the exponent range of fp32 and needs no shift.
template <bool KV>
struct BwdLayout {
    int panels, stages;
    __host__ __device__ int tile() const { return panels * kPanelBytes; }
    __host__ __device__ int ring() const { return 2 * tile(); }
    __host__ __device__ int aux() const { return ring() + stages * tile(); }  // per walked tile: lse and delta, or the mask
    __host__ __device__ int aux_bytes() const { return KV ? 2 * kRows * 4 : 16; }
    __host__ __device__ int bars() const { return aux() + stages / 2 * aux_bytes(); }
    __host__ __device__ int total() const { return bars() + 256 + 1024; }  // + alignment slack
};

constexpr int kBwdWarps = 8 + 1 + kLoadWarps;

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

template <typename T, int LG, bool ALIGNED, bool KV>
__global__ void __launch_bounds__(kBwdWarps * 32, 1) attn_bwd_mma(AttnArgs a, BwdLayout<KV> L) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ int s_dead;
    __shared__ uint32_t s_tmem;
    const AttnTile tl = KV ? attn_tile(a.k_off, a.graphs, 1, kRows, blockIdx.x) : attn_tile(a.q_off, a.graphs, a.group, kRows, blockIdx.x);
    if (tl.graph < 0) return;
    const int h = blockIdx.y, split = blockIdx.z;
    const int64_t q0 = a.q_off[tl.graph], k0 = a.k_off[tl.graph];
    const int64_t rows = (a.q_off[tl.graph + 1] - q0) * a.group, states = a.k_off[tl.graph + 1] - k0;
    const Piece walk = piece_of(KV ? rows : states, split, a.splits);
    const int n_tiles = int((walk.hi - walk.lo + kRows - 1) / kRows);
    const int own = int(min(tl.rows - tl.row0, int64_t(kRows)));  // rows of the resident tile
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int d16 = (a.D + 15) / 16, half = L.stages / 2;
    const uint32_t r_full = sb + L.bars(), s_full = r_full + 8, dp_full = s_full + 8, p_ready = dp_full + 8, ds_ready = p_ready + 8,
                   done = ds_ready + 8, fin = done + 8, full = fin + 8, empty = full + 8 * L.stages, aux_full = empty + 8 * L.stages;
    const uint32_t g_cols = uint32_t(64 * L.panels);
    const uint32_t tmem_cols = 512;
    if (threadIdx.x == 0) {
        s_dead = 0;
        bar_init(r_full, kLoadThreads);
        bar_init(s_full, 1);
        bar_init(dp_full, 1);
        bar_init(p_ready, 8);
        bar_init(ds_ready, 8);
        bar_init(done, 1);
        bar_init(fin, 1);
        for (int s = 0; s < L.stages; ++s) {
            bar_init(full + 8 * s, kLoadThreads);
            bar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < half; ++s) bar_init(aux_full + 8 * s, KV ? kLoadThreads : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) tmem_alloc(smem_u32(&s_tmem), tmem_cols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
    const uint32_t t_dp = tmem + kRows, t_g = tmem + 2 * kRows;  // sums: dq, or dk then dv
    volatile int* dead = &s_dead;
    unsigned* status = &attn_status_word;
    constexpr float kShift = __is_same(T, __half) ? 8.f : 0.f, kUnshift = __is_same(T, __half) ? 0.00390625f : 1.f;
    constexpr float kLog2e = 1.4426950408889634f;

    if (warp < 8) {
        // ----------------------------------------------------------------- P and dS
        const int w = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const bool work = quad * 32 < own;
        const uint32_t lanes = uint32_t(quad * 32) << 16, col = uint32_t(64 * w);
        const float c = a.scale_log2;
        const int64_t p = tl.row0 + row;
        float lse = INFINITY, delta = 0.f;  // of the thread's row (dq)
        int64_t rh = 0;
        bool keep = row < own;
        if (keep) {
            if (KV) {
                rh = (k0 + p) * a.Hkv + h;
                keep = !a.keep || a.keep[k0 + p];
            } else {
                rh = (q0 + p / a.group) * a.Hq + int64_t(h) * a.group + p % a.group;
                const float x = a.lse[rh];
                // a row without a kept state: P = exp2(s - inf) = 0
                lse = x == -INFINITY ? INFINITY : x * kLog2e - kShift;
                delta = a.delta[rh] * kUnshift;
            }
        }
        bool ok = true;
        for (int j = 0; j < n_tiles; ++j) {
            const int ax = j % half;
            const float* s_lse = reinterpret_cast<const float*>(smem + L.aux() + ax * L.aux_bytes()) + col;
            const float* s_delta = s_lse + kRows;
            uint32_t word[2] = {0xffffffffu, 0xffffffffu};
            if (KV || a.keep) {
                ok = __all_sync(0xffffffffu, bar_wait(aux_full + 8 * ax, (j / half) & 1, dead, status));
                if (!ok) break;
            }
            if (!KV) {
                if (a.keep) {
                    const uint32_t* mw = reinterpret_cast<const uint32_t*>(smem + L.aux() + ax * L.aux_bytes()) + 2 * w;
                    word[0] = mw[0];
                    word[1] = mw[1];
                } else {
                    const int64_t left = walk.hi - walk.lo - int64_t(j) * kRows;
                    word[0] = tail_word(left, 2 * w);
                    word[1] = tail_word(left, 2 * w + 1);
                }
            }
            ok = __all_sync(0xffffffffu, bar_wait(s_full, j & 1, dead, status));
            if (!ok) break;
            fence_after();
            float x[2][32];
            if (work) {
#pragma unroll
                for (int b = 0; b < 2; ++b) tmem_ld32(tmem + lanes + col + 32 * b, x[b]);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    tmem_wait_ld(x[b]);
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[b][i] = exp2_approx(fmaf(x[b][i], c, KV ? -s_lse[32 * b + i] : -lse));
                    if (!KV && word[b] != 0xffffffffu) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((word[b] >> i) & 1)) x[b][i] = 0.f;
                    }
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
            ok = __all_sync(0xffffffffu, bar_wait(dp_full, j & 1, dead, status));
            if (!ok) break;
            fence_after();
            if (work) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    float y[32];
                    tmem_ld32(t_dp + lanes + col + 32 * b, y);
                    tmem_wait_ld(y);
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[i] = x[b][i] * fmaf(y[i], kUnshift, KV ? -s_delta[32 * b + i] : -delta);
                    uint32_t q[16];
                    if (!KV && word[b] != 0xffffffffu) {  // 0 * (NaN - delta) is not 0
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!((word[b] >> i) & 1)) y[i] = 0.f;
                    }
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
            ok = __all_sync(0xffffffffu, bar_wait(done, 0, dead, status));
            fence_after();
        }
        if (ok && work) {
            // dk: warpgroup 0, dv: warpgroup 1; dq: the column blocks in turn
            const int64_t n = KV ? a.nk * a.Hkv : a.nq * a.Hq;
            T* dst = static_cast<T*>(KV ? (w ? a.dv : a.dk) : a.dq) + rh * a.D;
            float* part = a.splits > 1 ? a.part_o + ((KV && w ? a.splits + split : split) * n + rh) * a.D : nullptr;
            const bool vec = a.D % 8 == 0 && (reinterpret_cast<uintptr_t>(dst) & 15u) == 0;
            const float scale = KV && w ? kUnshift : a.scale;
            for (int d = KV ? 0 : w; d < d16; d += KV ? 1 : 2) {
                float o[16];
                __syncwarp();
                if (n_tiles > 0) {
                    tmem_ld16(t_g + lanes + (KV ? uint32_t(w) * g_cols : 0u) + 16 * d, o);
                    tmem_wait_ld(o);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = n_tiles > 0 && keep ? o[i] : 0.f;
                if (row < own) store_grad16<T>(o, scale, dst, part, 16 * d, a.D, vec);
            }
        }
    } else if (warp == 8) {
        // ----------------------------------------------------------------- matrix instructions
        if (lane == 0) {
            const uint32_t id_s = mma_desc<T>(kRows, false), id_g = mma_desc<T>(16 * d16, true);
            const uint32_t r1 = sb, r2 = sb + uint32_t(L.tile());
            auto stage = [&](int i) { return sb + uint32_t(L.ring() + (i % L.stages) * L.tile()); };
            auto wait_stage = [&](int i) {
                if (!bar_wait(full + 8 * (i % L.stages), (i / L.stages) & 1, dead, status)) return false;
                fence_async();
                return true;
            };
            auto product = [&](uint32_t d, uint32_t r, uint32_t x, uint32_t bar) {
                for (int s = 0; s < d16; ++s) mma_ss(d, desc_cols(r, s), desc_cols(x, s), id_s, s > 0);
                mma_commit(bar);
            };
            // d += A X: the 16-bit A of row block s lies in the half that its warpgroup wrote
            auto sum = [&](uint32_t d, uint32_t A, uint32_t x, bool first) {
#pragma unroll
                for (int s = 0; s < kRows / 16; ++s)
                    mma_ts(d, A + uint32_t((s >> 2) * 64 + (s & 3) * 8), desc_rows(x, s), id_g, !first || s > 0);
            };
            bool ok = n_tiles > 0 && bar_wait(r_full, 0, dead, status) && wait_stage(0);
            if (ok) {
                product(tmem, r1, stage(0), s_full);
                ok = wait_stage(1);
                if (ok) {
                    product(t_dp, r2, stage(1), dp_full);
                    if (!KV) mma_commit(empty + 8 * 1);
                }
            }
            for (int j = 0; j < n_tiles && ok; ++j) {
                ok = bar_wait(p_ready, j & 1, dead, status);
                if (!ok) break;
                fence_after();
                if (KV) {
                    sum(t_g + g_cols, tmem, stage(2 * j + 1), j == 0);
                    mma_commit(empty + 8 * ((2 * j + 1) % L.stages));
                }
                if (j + 1 < n_tiles) {
                    ok = wait_stage(2 * j + 2);
                    if (!ok) break;
                    product(tmem, r1, stage(2 * j + 2), s_full);
                }
                ok = bar_wait(ds_ready, j & 1, dead, status);
                if (!ok) break;
                fence_after();
                sum(t_g, t_dp, stage(2 * j), j == 0);
                mma_commit(empty + 8 * ((2 * j) % L.stages));
                if (j + 1 < n_tiles) {
                    ok = wait_stage(2 * j + 3);
                    if (!ok) break;
                    product(t_dp, r2, stage(2 * j + 3), dp_full);
                    if (!KV) mma_commit(empty + 8 * ((2 * j + 3) % L.stages));
                } else {
                    mma_commit(done);
                }
            }
            // every instruction issued has finished before the tensor memory and the stages go
            mma_commit(fin);
            bar_wait_last(fin, 0, status);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------------- loaders
        const int t = threadIdx.x - 9 * 32;
        const LoadMap<LG> map(t, a.D);
        if (n_tiles > 0) {
            auto arrive = [&](uint32_t bar) { ALIGNED ? copy_arrive(bar) : bar_arrive(bar); };
            const char* Q = reinterpret_cast<const char*>(static_cast<const T*>(a.q) + q0 * a.q_row + int64_t(h) * a.group * a.q_head);
            const char* dO = reinterpret_cast<const char*>(static_cast<const T*>(a.d_out) + q0 * a.o_row + int64_t(h) * a.group * a.o_head);
            const int64_t s0 = k0 + (KV ? tl.row0 : walk.lo);
            const char* K = reinterpret_cast<const char*>(static_cast<const T*>(a.k) + s0 * a.k_row + h * a.k_head) + map.chunk * 16;
            const char* V = reinterpret_cast<const char*>(static_cast<const T*>(a.v) + s0 * a.v_row + h * a.v_head) + map.chunk * 16;
            StateMask mask(a.keep ? a.keep + k0 : nullptr, KV ? tl.row0 : walk.lo, KV ? states : walk.hi);
            auto states_tile = [&](uint32_t dst, const char* src, int64_t stride) {
                auto use = [&](int r) { return mask.has(r); };
                if (mask.all())
                    load_strided<LG, ALIGNED, true>(dst, src, stride, map, use);
                else
                    load_strided<LG, ALIGNED, false>(dst, src, stride, map, use);
            };
            auto rows_tile = [&](uint32_t dst, const char* base, int64_t row, int64_t head, int64_t r0, int n) {
                load_packed<LG, ALIGNED>(dst, base, row * 2, head * 2, a.group, r0, n, map);
            };
            auto free_stage = [&](int i) {
                return i < L.stages || __all_sync(0xffffffffu, bar_wait(empty + 8 * (i % L.stages), (i / L.stages - 1) & 1, dead, status));
            };
            auto stage = [&](int i) { return sb + uint32_t(L.ring() + (i % L.stages) * L.tile()); };
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
            float v_lse[2], v_delta[2];
            auto fetch = [&](int j) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int64_t r = walk.lo + int64_t(j) * kRows + t + 64 * i;
                    v_lse[i] = -INFINITY, v_delta[i] = 0.f;
                    if (r < walk.hi) {
                        const int64_t q = r / a.group, at = (q0 + q) * a.Hq + int64_t(h) * a.group + (r - q * a.group);
                        v_lse[i] = a.lse[at];
                        v_delta[i] = a.delta[at];
                    }
                }
            };
            if (KV) fetch(0);
            for (int j = 0; j < n_tiles; ++j) {
                const int64_t lo = walk.lo + int64_t(j) * kRows;
                const int n = int(min(walk.hi - lo, int64_t(kRows)));
                if (!free_stage(2 * j)) break;
                // the tile that used this aux entry before gave up its X1 stage, which is this one
                if (KV) {
                    float* s_lse = reinterpret_cast<float*>(smem + L.aux() + (j % half) * L.aux_bytes());
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // rows past the end and rows without a kept state: P = exp2(s - inf) = 0
                        s_lse[t + 64 * i] = v_lse[i] == -INFINITY ? INFINITY : v_lse[i] * kLog2e - kShift;
                        s_lse[kRows + t + 64 * i] = v_delta[i] * kUnshift;
                    }
                    bar_arrive(aux_full + 8 * (j % half));
                    if (j + 1 < n_tiles) fetch(j + 1);
                    rows_tile(stage(2 * j), Q, a.q_row, a.q_head, lo, n);
                    arrive(full + 8 * ((2 * j) % L.stages));
                    if (!free_stage(2 * j + 1)) break;
                    rows_tile(stage(2 * j + 1), dO, a.o_row, a.o_head, lo, n);
                    arrive(full + 8 * ((2 * j + 1) % L.stages));
                } else {
                    mask.next();
                    if (a.keep && t == 0) {
                        *reinterpret_cast<uint4*>(smem + L.aux() + (j % half) * L.aux_bytes()) =
                            make_uint4(mask.word[0], mask.word[1], mask.word[2], mask.word[3]);
                        bar_arrive(aux_full + 8 * (j % half));
                    }
                    states_tile(stage(2 * j), K, a.k_row * 2);
                    arrive(full + 8 * ((2 * j) % L.stages));
                    if (!free_stage(2 * j + 1)) break;
                    states_tile(stage(2 * j + 1), V, a.v_row * 2);
                    arrive(full + 8 * ((2 * j + 1) % L.stages));
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

template <typename T, int LG, bool ALIGNED, bool KV>
cudaError_t bwd_lg(const AttnArgs& a, int64_t tiles, cudaStream_t st) {
    BwdLayout<KV> L;
    L.panels = a.D > 64 ? 2 : 1;
    L.stages = L.panels == 1 ? 8 : 4;  // 160 or 192 KB
    auto k = attn_bwd_mma<T, LG, ALIGNED, KV>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L.total());
    if (e != cudaSuccess) return e;
    k<<<dim3(unsigned(tiles), unsigned(a.Hkv), unsigned(a.splits)), kBwdWarps * 32, L.total(), st>>>(a, L);
    return cudaGetLastError();
}
template <typename T, bool ALIGNED, bool KV>
cudaError_t bwd(const AttnArgs& a, int64_t tiles, cudaStream_t st) {
    if (a.D <= 16) return bwd_lg<T, 1, ALIGNED, KV>(a, tiles, st);
    if (a.D <= 32) return bwd_lg<T, 2, ALIGNED, KV>(a, tiles, st);
    if (a.D <= 64) return bwd_lg<T, 3, ALIGNED, KV>(a, tiles, st);
    return bwd_lg<T, 4, ALIGNED, KV>(a, tiles, st);
}
template <typename T>
cudaError_t bwd_of(const AttnArgs& a, bool kv, int64_t tiles, cudaStream_t st) {
    const uintptr_t any = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                          reinterpret_cast<uintptr_t>(a.d_out) |
                          uintptr_t(a.q_row | a.q_head | a.k_row | a.k_head | a.v_row | a.v_head | a.o_row | a.o_head) * 2;
    if (any & 15u) return kv ? bwd<T, false, true>(a, tiles, st) : bwd<T, false, false>(a, tiles, st);
    return kv ? bwd<T, true, true>(a, tiles, st) : bwd<T, true, false>(a, tiles, st);
}

template <typename T, int NT, int LG, bool ALIGNED>
cudaError_t fwd_lg(const AttnArgs& a, int64_t row_tiles, cudaStream_t st) {
    FwdLayout<NT> L;
    L.panels = a.D > 64 ? 2 : 1;
    // one panel: 96 KB, two CTAs per SM (NT = 1), or 160 KB; two panels: 224 KB
    L.stages = NT == 1 ? (L.panels == 1 ? 5 : 6) : (L.panels == 1 ? 8 : 5);
    auto k = attn_fwd_mma<T, NT, LG, ALIGNED>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L.total());
    if (e != cudaSuccess) return e;
    k<<<dim3(unsigned(row_tiles), unsigned(a.Hkv), unsigned(a.splits)), (4 * NT + 1 + kLoadWarps) * 32, L.total(), st>>>(a, L);
    return cudaGetLastError();
}

template <typename T, int NT, bool ALIGNED>
cudaError_t fwd(const AttnArgs& a, int64_t row_tiles, cudaStream_t st) {
    if (a.D <= 16) return fwd_lg<T, NT, 1, ALIGNED>(a, row_tiles, st);
    if (a.D <= 32) return fwd_lg<T, NT, 2, ALIGNED>(a, row_tiles, st);
    if (a.D <= 64) return fwd_lg<T, NT, 3, ALIGNED>(a, row_tiles, st);
    return fwd_lg<T, NT, 4, ALIGNED>(a, row_tiles, st);
}
template <typename T>
cudaError_t fwd_of(const AttnArgs& a, int nt, int64_t row_tiles, cudaStream_t st) {
    const uintptr_t any = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                          uintptr_t(a.q_row | a.q_head | a.k_row | a.k_head | a.v_row | a.v_head) * 2;
    if (any & 15u) return nt == 2 ? fwd<T, 2, false>(a, row_tiles, st) : fwd<T, 1, false>(a, row_tiles, st);
    return nt == 2 ? fwd<T, 2, true>(a, row_tiles, st) : fwd<T, 1, true>(a, row_tiles, st);
}

}  // namespace

cudaError_t launch_attn_fwd_mma(uvu_dtype dtype, const AttnArgs& a, int nt, int64_t row_tiles, cudaStream_t st) {
    return dtype == UVU_BF16 ? fwd_of<__nv_bfloat16>(a, nt, row_tiles, st) : fwd_of<__half>(a, nt, row_tiles, st);
}

cudaError_t launch_attn_bwd_mma(uvu_dtype dtype, const AttnArgs& a, bool kv, int64_t tiles, cudaStream_t st) {
    return dtype == UVU_BF16 ? bwd_of<__nv_bfloat16>(a, kv, tiles, st) : bwd_of<__half>(a, kv, tiles, st);
}

// Status of the tensor-core attention kernels on the current device (bit 0: a bounded wait gave up).
cudaError_t attn_status(unsigned* word, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(word, attn_status_word, sizeof(unsigned));
    if (e != cudaSuccess || !reset) return e;
    const unsigned z = 0;
    return cudaMemcpyToSymbol(attn_status_word, &z, sizeof(unsigned));
}

}  // namespace uvu
