// What the tensor-core attention kernels share: loading of operand tiles, masks, the split of a walk.
//
// The loaders use 16-byte cp.async with zero fill instead of tensor maps: a masked or absent state is
// zeros in shared memory, whatever memory holds there (0 * NaN would reach a sum), and any row and head
// strides work; operands off the 16-byte grid go through registers.  A stage's barrier counts the
// loader threads, whose arrivals are tied to their copies; the issuer of the matrix instructions orders
// what they wrote before its instructions (a proxy fence after the barrier).
//
// Every wait is bounded (two seconds); on expiry the roles leave their loops, the issuer waits for its
// instructions, the loaders for their copies, and the CTA frees its tensor memory and returns with the
// status word set.
#pragma once

#include <algorithm>
#include <cstdint>

#include "attn.h"
#include "elem.h"
#include "tensor_core.h"

namespace uvu {
namespace {

using namespace tc;

__device__ unsigned int attn_status_word;  // of the including file's kernels; see attn_status()

// The word of this file's kernels (bit 0: a bounded wait gave up); reset clears it.
cudaError_t read_status(unsigned* word, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(word, attn_status_word, sizeof(unsigned));
    if (e != cudaSuccess || !reset) return e;
    const unsigned z = 0;
    return cudaMemcpyToSymbol(attn_status_word, &z, sizeof(unsigned));
}

constexpr int kRows = 128;      // rows of a row tile, states of a state tile
constexpr int kLoadWarps = 2;   // where nothing else is said
constexpr float kLn2 = 0.6931471805599453f;

constexpr int kLoadThreads = kLoadWarps * 32;

// How the loader threads share a tile of ROWS rows: thread t takes 16-byte chunk t % 2^LG of the rows
// t / 2^LG, + kStep, ...  2^LG is the power of two that holds the row's chunks.
template <int LG, int ROWS_ = kRows, int THREADS = kLoadThreads>
struct LoadMap {
    static constexpr int ROWS = ROWS_, kStep = THREADS >> LG, kIters = ROWS / kStep;
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

// A tile of rows, the thread's own `step` bytes apart from p on; those that use(i) refuses are zeros.  ALL: every row is used.
template <bool ALIGNED, bool ALL, typename M, typename Use>
__device__ __forceinline__ void load_rows(uint32_t dst, const char* p, int64_t step, const M& m, Use use) {
    if (!m.on) return;
    // rows kStep apart share their swizzle when kStep is a multiple of 8; at 4 it alternates
    const uint32_t even = dst + tile_offset(m.row, m.chunk), odd = dst + tile_offset(m.row + M::kStep, m.chunk) - uint32_t(M::kStep * 128);
#pragma unroll 8
    for (int i = 0; i < M::kIters; ++i) {
        load_chunk<ALIGNED>((i & 1 ? odd : even) + uint32_t(i * M::kStep * 128), p, ALL || use(i) ? m.bytes : 0);
        p += step;
    }
}

// Packed rows of a kv head's queries from r0 on: row r is query r / group, head r % group.  Rows from `rows` on are
// zeros, or left alone (!ZERO: rows of the M side, whose lanes nobody reads).
template <bool ALIGNED, bool ZERO, typename M>
__device__ __forceinline__ void load_packed(uint32_t dst, const char* base, int64_t row, int64_t head, int group, int64_t r0, int rows,
                                            const M& m) {
    if (!m.on) return;
    // query and head of the thread's first row; later rows step by kStep without a division
    const uint32_t g = uint32_t(group), dq = g == 1 ? uint32_t(M::kStep) : uint32_t(M::kStep) / g, dj = uint32_t(M::kStep) - dq * g;
    const int64_t q0 = group == 1 ? r0 + m.row : (r0 + m.row) / group;
    uint32_t j = uint32_t(r0 + m.row - q0 * group);
    const char* p = base + q0 * row + int64_t(j) * head + m.chunk * 16;
    // the group divides kStep (1, 2, 4 of 4 to 32): the thread's rows are all of one head, a constant stride apart
    if (dj == 0 && (ZERO || rows >= M::ROWS)) {
        auto use = [&](int i) { return m.row + i * M::kStep < rows; };
        if (rows >= M::ROWS)
            load_rows<ALIGNED, true>(dst, p, dq * row, m, use);
        else
            load_rows<ALIGNED, false>(dst, p, dq * row, m, use);
        return;
    }
    const int64_t step = dq * row + int64_t(dj) * head, wrap = row - int64_t(g) * head;
#pragma unroll 4
    for (int i = 0; i < M::kIters; ++i) {
        const int r = m.row + i * M::kStep;
        if (!ZERO && r >= rows) break;
        load_chunk<ALIGNED>(dst + tile_offset(r, m.chunk), p, r < rows ? m.bytes : 0);
        p += step;
        j += dj;
        if (j >= g) {
            j -= g;
            p += wrap;
        }
    }
}

// A thread's packed rows r, r + step, ... of a kv head, and where their statistics are ([queries][heads]; `first`: of the
// first query's first head), without a division after the first row.
struct RowWalk {
    int64_t r, at, next_at;
    uint32_t j, g, dj, step;
    int heads;
    __device__ __forceinline__ RowWalk(int64_t row, int group, int64_t first, int heads_, int step_) : r(row), g(group), step(step_), heads(heads_) {
        const int64_t q = r / group;
        j = uint32_t(r - q * group);
        at = first + q * heads + j;
        dj = step % g;
        next_at = int64_t(step / g) * heads + dj;
    }
    __device__ __forceinline__ void next() {
        r += step;
        at += next_at;
        j += dj;
        if (j >= g) {
            j -= g;
            at += heads - int64_t(g);
        }
    }
};

__device__ __forceinline__ uint32_t tail_word(int64_t left, int w) {  // bits of the states that exist
    const int64_t n = left - 32 * w;
    return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << uint32_t(n)) - 1u;
}

// Which of a tile's N states take part, as words in every lane of a loader warp.  The mask bytes of
// the next tile are fetched a tile ahead.
template <int N = kRows>
struct StateMask {
    static constexpr int kWords = N / 32;
    const uint8_t* keep;  // of the graph, or null
    int64_t at, hi;       // first state of the coming tile, end
    uint32_t word[kWords], ahead;
    __device__ __forceinline__ StateMask(const uint8_t* k, int64_t lo, int64_t end) : keep(k), at(lo), hi(end), ahead(0) { fetch(); }
    __device__ __forceinline__ void fetch() {
        if (!keep) return;
        ahead = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const int64_t s = at + 32 * w + (threadIdx.x & 31);
            if (s < hi && keep[s]) ahead |= 1u << w;
        }
    }
    __device__ __forceinline__ void next() {
#pragma unroll
        for (int w = 0; w < kWords; ++w) word[w] = keep ? __ballot_sync(0xffffffffu, (ahead >> w) & 1) : tail_word(hi - at, w);
        at += N;
        fetch();
    }
    __device__ __forceinline__ bool all() const {
        uint32_t a = 0xffffffffu;
#pragma unroll
        for (int w = 0; w < kWords; ++w) a &= word[w];
        return a == 0xffffffffu;
    }
    __device__ __forceinline__ bool any() const {
        uint32_t a = 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) a |= word[w];
        return a != 0;
    }
    // The states row, row + STEP, ... (row < STEP) as the bits 0, 1, ... of a word.
    template <int STEP>
    __device__ __forceinline__ uint32_t every(int row) const {
        static_assert(STEP >= 4 && STEP <= 64 && N / STEP <= 32, "fits one word");
        constexpr int kWord = STEP < 32 ? 32 / STEP : 1;  // bits from a word
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < (N + STEP - 1) / STEP; i += kWord) {
            const int w = i * STEP / 32;
            uint32_t x = (STEP == 64 && row >= 32 ? word[w + 1 < kWords ? w + 1 : w] : word[w]) >> (row & 31);
            // groups of n bits STEP n apart join in pairs
            if constexpr (STEP == 4) x &= 0x11111111u, x = (x | x >> 3) & 0x03030303u, x = (x | x >> 6) & 0x000f000fu, x = x | x >> 12;
            if constexpr (STEP == 8) x &= 0x01010101u, x = (x | x >> 7) & 0x00030003u, x = x | x >> 14;
            if constexpr (STEP == 16) x &= 0x00010001u, x = x | x >> 15;
            mine |= (x & ((1u << kWord) - 1)) << i;
        }
        return mine;
    }
    __device__ __forceinline__ bool has(int r) const {
        uint32_t x = word[0];
#pragma unroll
        for (int w = 1; w < kWords; ++w) x = r >= 32 * w ? word[w] : x;
        return (x >> (r & 31)) & 1;
    }
};

// Writes 0 or -inf per state of the tile to `bias` (shared memory), by all loader threads.
template <int THREADS = kLoadThreads, int N>
__device__ __forceinline__ void write_bias(float* bias, const StateMask<N>& m, int t) {
#pragma unroll
    for (int i = 0; i < (N + THREADS - 1) / THREADS; ++i) {
        const int r = t + i * THREADS;
        if (r < N) bias[r] = m.has(r) ? 0.f : -INFINITY;
    }
}
// N columns plus a tile's bias from shared memory (16-byte aligned): masked columns become -inf.
template <int N>
__device__ __forceinline__ void add_bias(float (&v)[N], const float* bias) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        const ulonglong2 q = reinterpret_cast<const ulonglong2*>(bias)[i];
        F2 b0, b1;
        b0.v = q.x, b1.v = q.y;
        const float2 x = (F2(v[4 * i], v[4 * i + 1]) + b0).both(), y = (F2(v[4 * i + 2], v[4 * i + 3]) + b1).both();
        v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = y.x, v[4 * i + 3] = y.y;
    }
}
template <int N>
__device__ __forceinline__ float row_max(const float (&v)[N]) {
    float a = max3(v[0], v[1], v[2]), b = max3(v[3], v[4], v[5]);
#pragma unroll
    for (int i = 6; i + 1 < N; i += 4) {
        a = max3(a, v[i], v[i + 1]);
        if (i + 3 < N) b = max3(b, v[i + 2], v[i + 3]);
    }
    return fmaxf(a, b);
}
// v = exp2(c v - base), and the values' sum by pairs.
template <int N>
__device__ __forceinline__ void exp_row(float (&v)[N], F2 c, F2 minus, F2 (&sum)[2]) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float2 e = fma2(F2(v[2 * i], v[2 * i + 1]), c, minus).both();
        v[2 * i] = exp2_approx(e.x), v[2 * i + 1] = exp2_approx(e.y);
        sum[i & 1] = sum[i & 1] + F2(v[2 * i], v[2 * i + 1]);
    }
}

// The two steps of the backward on N columns of a row.  p = exp2(c s + e), then p (dp u - delta); e and delta are the
// row's, or per column (shared memory, 16-byte aligned; PER).
template <bool PER, int N>
__device__ __forceinline__ void bwd_p(float (&s)[N], F2 c, float e, const float* es) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        F2 add(e, e);
        if constexpr (PER) add.v = reinterpret_cast<const uint64_t*>(es)[i];
        const float2 x = fma2(F2(s[2 * i], s[2 * i + 1]), c, add).both();
        s[2 * i] = exp2_approx(x.x), s[2 * i + 1] = exp2_approx(x.y);
    }
}
template <bool PER, int N>
__device__ __forceinline__ void bwd_ds(float (&dp)[N], const float (&p)[N], F2 u, float minus_delta, const float* minus_deltas) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        F2 add(minus_delta, minus_delta);
        if constexpr (PER) add.v = reinterpret_cast<const uint64_t*>(minus_deltas)[i];
        const float2 x = (F2(p[2 * i], p[2 * i + 1]) * fma2(F2(dp[2 * i], dp[2 * i + 1]), u, add)).both();
        dp[2 * i] = x.x, dp[2 * i + 1] = x.y;
    }
}

// A tile of states with a constant stride, `src` the first (the thread's chunk included); those that take no part are zeros.
template <bool ALIGNED, typename M>
__device__ __forceinline__ void load_states(uint32_t dst, const char* src, int64_t stride, const M& m, const StateMask<M::ROWS>& mask) {
    const uint32_t mine = mask.template every<M::kStep>(m.row);
    if (mask.all())
        load_rows<ALIGNED, true>(dst, src + m.row * stride, M::kStep * stride, m, [](int) { return true; });
    else
        load_rows<ALIGNED, false>(dst, src + m.row * stride, M::kStep * stride, m, [&](int i) { return (mine >> i) & 1; });
}

// The stages of a ring in the order of their uses, without a division (by a variable it costs as much as several matrix
// instructions).
struct Ring {
    int n, at = 0, uses = 0;
    uint32_t parity = 0;  // of the use's phase
    __device__ __forceinline__ explicit Ring(int stages) : n(stages) {}
    __device__ __forceinline__ void next() {
        ++uses;
        if (++at == n) at = 0, parity ^= 1;
    }
};

struct Piece {
    int64_t lo, hi;
};
__device__ __forceinline__ Piece piece_of(int64_t n, int s, int splits) {
    const int64_t tiles = (n + kRows - 1) / kRows, per = (tiles + splits - 1) / splits;
    return {min(n, s * per * kRows), min(n, (s + 1) * per * kRows)};
}

// f(dimension class, aligned) for a head dimension: 2^class 16-byte chunks a row.  Operands off the
// 16-byte grid are rare and take one class for all dimensions.
template <typename F>
cudaError_t by_chunks(int D, bool aligned, F f) {
    if (!aligned) return f(std::integral_constant<int, 4>{}, std::false_type{});
    if (D <= 16) return f(std::integral_constant<int, 1>{}, std::true_type{});
    if (D <= 32) return f(std::integral_constant<int, 2>{}, std::true_type{});
    if (D <= 64) return f(std::integral_constant<int, 3>{}, std::true_type{});
    return f(std::integral_constant<int, 4>{}, std::true_type{});
}

}  // namespace
}  // namespace uvu
