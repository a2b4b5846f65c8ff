// Orthogonalised updates by Newton-Schulz products.
//
//     X_0 = G / (|G|_F + eps),   P = X X^T,   X <- a X + (b P + c P P) X,   out = scale X after `steps` of them
//
// on the side of the smaller Gram matrix (a tall G is turned): m <= n.  With M = a I + b P + c P P a step is three products,
// P = X X^T, P P and M X; the first two are symmetric, and only their lower blocks are formed.
//
// Products of fp32 accuracy on the 16-bit tensor cores: a value v is held as hi = fp16(v) and lo = fp16(2^11 (v - hi)), 22 bits
// and a sign, and hi hi + 2^-11 (hi lo + lo hi) is formed in two fp32 accumulators; lo lo (2^-24 of the product) is left out.  Errors
// matter here: a step stretches what is small in X by a = 3.4, five of them by 485, so 16-bit operands alone would be off by 1%
// and more where few singular values hold most of a gradient.  Values are held at 2^8 times their size, which keeps
// those of large matrices (1 / sqrt(m n)) normal numbers of fp16 and those near 1 far from its largest.  Below 2^-22 the bits get fewer, to an
// error of 2^-44: that matters where a gradient's norm lies far below eps.
//
// An accumulating matrix instruction (16 terms) cuts its sum towards zero, by 2^-24 of it in the mean (measured: 2.8 2^-24 after
// four of them, 7.7 after eight, on sums of one sign).  So the hi hi sums leave their accumulator every 64 terms, while the lo products,
// two thirds of the instructions, run (on chip they go to three accumulators in turn), and the mean of what was cut is put back: a
// factor 1 + 2^-24 for each instruction.  Five steps on 64 x 1664 values are off by 8e-7, by 2.4e-6 without all that; fp32 sums: 9.6e-7.
//
// A matrix is kept in panels of 128 rows and 64 columns, 16 KB each, whose bytes lie as the matrix instruction reads them
// (128-byte swizzle): a panel is loaded by one bulk copy, and no tensor map is needed.
//
// Two forms.  On chip, for m <= 128 and n <= 2048: a block, or a cluster of up to 8 that splits the columns, keeps X and P in shared
// memory from the first step to the last; one launch.  Else a kernel for each product, of tiles of 128 rows and 256, 128 or 64 columns.
//
// What bounds it.  Large matrices: the tensor cores (two of 4096 x 2048 in fp32: 1.27 to 1.42 ms, 1.42 to 1.27 PFLOP/s of fp16 products with a step
// of 250 us at first and 290 us when the card's power limit has lowered its clocks).  Small ones: the chain of three products a step, each of
// which waits for the last one's planes: some 2000 cycles of products of 128 x 128 x 128 and 2300 of writing planes on chip (13 of
// 128 x 128: 40 us; one of 64 x 1664 over a cluster of 8: 56 us), 9000 to 14,000 with loads and a launch otherwise (25 of 256 x 256 in bf16:
// 97 us).  One rolled loop in place of the three products' code on chip took 48 us: fetching costs in the first step alone.  All phases in one launch whose blocks
// wait for one another's tiles took as long: the flags cost what the launches do.
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "elem.h"
#include "plan.h"
#include "tensor_core.h"

namespace uvu {
namespace {

namespace cg = cooperative_groups;
using namespace tc;

__device__ unsigned int ortho_status_word;

constexpr int kPanel = 16384;  // bytes of a panel
constexpr float kHeld = 256.f, kHeldInv = 1.f / 256.f;  // values are held at this size
constexpr float kLo = 2048.f, kLoInv = 1.f / 2048.f;

// What makes good the mean cut of a sum by so many accumulating instructions.
__device__ __forceinline__ float uncut(int instructions) { return 1.f + float(instructions) * 0x1p-24f; }

__device__ __forceinline__ void arrive_tx(uint32_t b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
// Launches that follow one another: the next kernel's blocks may begin where there is room, and wait here for this one's end.
__device__ __forceinline__ void next_may_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Ordinary writes, of this block's shared memory or another's, come before asynchronous reads.
__device__ __forceinline__ void fence_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Two values' halves, each pair with the first value in the low half.
__device__ __forceinline__ void split(float v0, float v1, uint32_t& hi, uint32_t& lo) {
    hi = pack2<__half>(v0, v1);
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    const float2 r = fma2(F2(h.x, h.y), F2(-kLo, -kLo), F2(v0, v1) * F2(kLo, kLo)).both();
    lo = pack2<__half>(r.x, r.y);
}
// Eight values' halves: the 16 bytes of each plane.
struct Chunk {
    uint32_t hi[4], lo[4];
    __device__ __forceinline__ explicit Chunk(const float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) split(v[2 * i], v[2 * i + 1], hi[i], lo[i]);
    }
    __device__ __forceinline__ Chunk(const char* at, size_t plane) {
        const uint4 h = *reinterpret_cast<const uint4*>(at), l = *reinterpret_cast<const uint4*>(at + plane);
        hi[0] = h.x, hi[1] = h.y, hi[2] = h.z, hi[3] = h.w, lo[0] = l.x, lo[1] = l.y, lo[2] = l.z, lo[3] = l.w;
    }
    __device__ __forceinline__ void store(char* at, size_t plane) const {
        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + plane) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    __device__ __forceinline__ float value(int i) const {
        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi[i >> 1])),
                     l = __half22float2(*reinterpret_cast<const __half2*>(&lo[i >> 1]));
        return i & 1 ? fmaf(l.y, kLoInv, h.y) : fmaf(l.x, kLoInv, h.x);
    }
};
// A shared-memory address for an operand's descriptor, which has room for the offset in the block's own memory alone: in a cluster the
// address also has the block's rank, in its upper byte.
__device__ __forceinline__ uint32_t own_offset(uint32_t address) { return address & 0x3FFFFu; }
// Where a panel holds row r (of its 128) and column c (of its 64).
__device__ __forceinline__ uint32_t in_panel(int r, int c) {
    return uint32_t((r >> 3) * 1024 + (r & 7) * 128 + ((((c >> 3) ^ r) & 7) << 4) + (c & 7) * 2);
}

// The squares' sum of values of any size, in fp32: those of large and of small values at scales of their own.  (The card has little fp64:
// one thread of a block uses it, at the end.)
struct Squares {
    float small = 0.f, mid = 0.f, large = 0.f;
    __device__ __forceinline__ void add(float v) {
        v = fabsf(v);
        if (v > 0x1p50f) {
            v *= 0x1p-90f;
            large = fmaf(v, v, large);
        } else if (v < 0x1p-50f) {
            v *= 0x1p90f;
            small = fmaf(v, v, small);
        } else {
            mid = fmaf(v, v, mid);  // a NaN comes here
        }
    }
    // N values at once, at one scale where nothing that counts is lost below 2^-126 or overflows
    template <int N>
    __device__ __forceinline__ void add_all(const float (&v)[N]) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) sum = fmaf(v[i], v[i], sum);
        if (sum > 0x1p-60f && sum < 0x1p100f) {
            mid += sum;
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) add(v[i]);
        }
    }
    __device__ __forceinline__ void over_warp() {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            small += __shfl_xor_sync(0xffffffffu, small, d);
            mid += __shfl_xor_sync(0xffffffffu, mid, d);
            large += __shfl_xor_sync(0xffffffffu, large, d);
        }
    }
    __device__ __forceinline__ void add(const Squares& o) { small += o.small, mid += o.mid, large += o.large; }
};
// Over the block, in thread 0.
template <int WARPS>
__device__ __forceinline__ Squares block_squares(Squares q) {
    __shared__ Squares s_part[WARPS];
    q.over_warp();
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = q;
    __syncthreads();
    q = threadIdx.x < WARPS ? s_part[threadIdx.x] : Squares();
    if (threadIdx.x < 32) q.over_warp();
    return q;
}

// X's rows and columns, and where the caller's matrix has them: X[r][c] at r * row + c, or at c * row + r where it is turned.
struct Side {
    int m, n;
    bool turned;
    int64_t matrix, row;
};

// ------------------------------------------------------------------------------- norm and planes

constexpr int kNormBlocks = 256;  // partial sums of a matrix at most

// V consecutive values at p where all V are inside, else those below `left`; zeros beyond.
template <typename T, int V>
__device__ __forceinline__ void load_some(const T* p, int left, bool vec, float (&v)[V]) {
    if (vec && left >= V) {
        constexpr int kEach = 16 / int(sizeof(T));
#pragma unroll
        for (int i = 0; i < V / kEach; ++i) {
            const Vec<T, kEach> q = load_vec<T, kEach>(p + i * kEach);
#pragma unroll
            for (int k = 0; k < kEach; ++k) v[i * kEach + k] = widen(q.v[k]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < left ? widen(p[i]) : 0.f;
    }
}

// 8 values of a row a thread, 4 times at once.
template <typename T>
__global__ void __launch_bounds__(256) norm_kernel(int rows, int cols, int64_t g_matrix, int64_t g_row, bool vec, const T* g, Squares* part) {
    const T* a = g + int64_t(blockIdx.y) * g_matrix;
    const int chunks = (cols + 7) / 8;
    const int count = rows * chunks;
    Squares q;
    for (int i0 = blockIdx.x * 1024; i0 < count; i0 += gridDim.x * 1024) {
        float v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * 256 + int(threadIdx.x), r = i / chunks, c = (i - r * chunks) * 8;
            load_some<T, 8>(a + (i < count ? r * g_row + c : 0), i < count ? cols - c : 0, vec, v[u]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) q.add_all(v[u]);
    }
    const Squares total = block_squares<8>(q);
    if (threadIdx.x == 0) part[blockIdx.y * kNormBlocks + blockIdx.x] = total;
}

// The factor 1 / (|G| + eps), as two: fp32 does not hold the inverse of the smallest norms, nor all bits of that of the largest.  Zeros
// stay zeros, with eps = 0 too; an infinity makes the whole matrix NaN, as a NaN does.
struct Factor {
    float first, second;
    __device__ __forceinline__ Factor() {}
    __device__ __forceinline__ Factor(const Squares& q, double eps) {
        first = 1.f;
        if (q.small < 0x1p100f && q.large == 0.f && q.mid > 0x1p-60f && q.mid < 0x1p120f && eps < 0x1p100) {  // what `small` stands for is below 2^-80
            second = 1.f / (sqrtf(q.mid) + float(eps));
        } else {  // rarely: fp64 is slow here
            const double squares = double(q.small) * 0x1p-180 + double(q.mid) + double(q.large) * 0x1p180;
            const double inv = squares == 0.0 ? 0.0 : isinf(squares) ? double(NAN) : 1.0 / (sqrt(squares) + eps);
            if (inv > 0x1p100) first = 0x1p60f;
            if (inv < 0x1p-100) first = 0x1p-60f;
            second = float(inv / double(first));
        }
    }
    __device__ __forceinline__ float of(float v) const { return v * first * second; }
};

// That of the block's matrix, in every thread of the block.
__device__ __forceinline__ Factor inverse_norm(const Squares* part, int parts, double eps) {
    __shared__ Factor s_inv;
    if (threadIdx.x < 32) {
        Squares q;
        for (int i = threadIdx.x; i < parts; i += 32) q.add(part[i]);
        q.over_warp();
        if (threadIdx.x == 0) s_inv = Factor(q, eps);
    }
    __syncthreads();
    return s_inv;
}

// X_0's planes, a 64 x 64 piece a block: (column panel, half a row block, matrix).
template <typename T>
__global__ void __launch_bounds__(256) take_kernel(Side s, bool vec, const T* g, const Squares* part, int parts, double eps, int panels,
                                                   size_t plane, char* x) {
    __shared__ float tile[64][65];
    const T* a = g + int64_t(blockIdx.z) * s.matrix;
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
    // 8 values that are consecutive in G: of row u of the piece, or of the turned one's column u
    const int u = threadIdx.x >> 3, first = (threadIdx.x & 7) * 8;
    float v[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int line = (s.turned ? c0 : r0) + u + 32 * i, at = (s.turned ? r0 : c0) + first;
        const bool live = line < (s.turned ? s.n : s.m);
        load_some<T, 8>(a + (live ? line * s.row + at : 0), live ? (s.turned ? s.m : s.n) - at : 0, vec, v[i]);
    }
    const Factor inv = inverse_norm(part + int64_t(blockIdx.z) * kNormBlocks, parts, eps);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = inv.of(v[i][k]) * kHeld;
    if (s.turned) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) tile[u + 32 * i][first + k] = v[i][k];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = tile[first + k][u + 32 * i];
    }
    char* to = x + int64_t(blockIdx.z) * 2 * plane + (int64_t(blockIdx.y >> 1) * panels + blockIdx.x) * kPanel;
#pragma unroll
    for (int i = 0; i < 2; ++i) Chunk(v[i]).store(to + in_panel((blockIdx.y & 1) * 64 + u + 32 * i, first), plane);
}

// No steps: out = scale X_0.
template <typename T>
__global__ void __launch_bounds__(256) scale_kernel(int rows, int cols, int64_t g_matrix, int64_t g_row, int64_t o_matrix, int64_t o_row,
                                                    float scale, const T* g, const Squares* part, int parts, double eps, T* out) {
    const Factor inv = inverse_norm(part + int64_t(blockIdx.y) * kNormBlocks, parts, eps);
    const T* a = g + int64_t(blockIdx.y) * g_matrix;
    T* o = out + int64_t(blockIdx.y) * o_matrix;
    for (int r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < cols; c += blockDim.x) o[r * o_row + c] = narrow<T>(inv.of(widen(a[r * g_row + c])) * scale);
}

// A tile of fp32 sums in shared memory, [rows][width], on its way to panels or to the caller's matrix: rows and columns of it are read
// by other threads than wrote them, so that global memory is written in whole lines.  The 16-byte chunks of a row are exchanged by its
// number, so that neither direction meets bank conflicts (width is a multiple of 64).
__device__ __forceinline__ int in_stage(int r, int chunk, int width) { return r * width + ((chunk ^ ((r ^ (r >> 3)) & 15)) << 2); }
template <int N>
__device__ __forceinline__ void stage(float* to, int r, int c, int width, const float (&v)[N]) {
#pragma unroll
    for (int k = 0; k < N / 4; ++k)
        *reinterpret_cast<float4*>(to + in_stage(r, c / 4 + k, width)) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
}
// Columns 8 k .. 8 k + 7 of row r, and rows 8 k .. 8 k + 7 of column c.
__device__ __forceinline__ void staged_row(const float* from, int r, int k, int width, float (&v)[8]) {
    const float4 x = *reinterpret_cast<const float4*>(from + in_stage(r, 2 * k, width)),
                 y = *reinterpret_cast<const float4*>(from + in_stage(r, 2 * k + 1, width));
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}
__device__ __forceinline__ void staged_column(const float* from, int c, int k, int width, float (&v)[8]) {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = from[in_stage(8 * k + q, c >> 2, width) + (c & 3)];
}
// The first `left` of eight values, which lie together.
template <typename T>
__device__ __forceinline__ void give8(T* o, int left, bool vec, const float (&v)[8]) {
    if (vec && left >= 8) {
        constexpr int kEach = 16 / int(sizeof(T));
#pragma unroll
        for (int b = 0; b < 8 / kEach; ++b) {
            Vec<T, kEach> q;
#pragma unroll
            for (int e = 0; e < kEach; ++e) q.v[e] = narrow<T>(v[b * kEach + e]);
            store_vec<T, kEach>(o + b * kEach, q);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < left) o[e] = narrow<T>(v[e]);
    }
}
// By `threads` threads: rows r0 .. r0 + 127 and columns c0 .. c0 + width - 1 of X, along what is consecutive in the caller's matrix.
template <typename T>
__device__ __forceinline__ void give(const float* from, int threads, const Side& s, T* out, bool vec, int r0, int c0, int width) {
    const int chunks = s.turned ? 16 : width / 8;
    const int lines = s.turned ? min(width, s.n - c0) : min(128, s.m - r0);
    const int step = threads / chunks, rest = threads - step * chunks;
    int line = int(threadIdx.x) / chunks, k = int(threadIdx.x) - line * chunks;
#pragma unroll 1
    for (; line < lines; line += step, k += rest) {
        if (k >= chunks) {
            k -= chunks;
            if (++line >= lines) break;
        }
        float v[8];
        if (s.turned) {
            staged_column(from, line, k, width, v);
            give8<T>(out + (c0 + line) * s.row + r0 + 8 * k, s.m - r0 - 8 * k, vec, v);
        } else {
            staged_row(from, line, k, width, v);
            give8<T>(out + (r0 + line) * s.row + c0 + 8 * k, s.n - c0 - 8 * k, vec, v);
        }
    }
}

// ------------------------------------------------------------------------------------ one product

enum Kind { kGram, kSquare, kApply, kLast };

struct Product {
    const char *A, *B, *own;  // panels of 128 rows (B of kApply: the rows are the summed index); own: P of kSquare where b is not 0
    char* out;
    size_t a_plane, b_plane, o_plane;      // bytes of a plane; a matrix has two
    int a_panels, b_panels, o_panels;      // of a row block
    int blocks;                            // row blocks of the result
    int k_panels;                          // of 64 summed values
    int tiles;                             // of a matrix
    int m;
    float diagonal, b, c;                  // kGram: P + diagonal I; kSquare: c P P + b P + diagonal I
    // kLast
    Side side;
    float scale;
    bool vec;
    void* result;
};

constexpr int kSumWarps = 16;  // they add up and write; then one that loads, and one that issues the matrix instructions
constexpr int kThreads = (kSumWarps + 2) * 32;
constexpr int kMaxSplits = 8;  // of a long sum

template <int BN>
struct Tile {
    static constexpr int a_bytes = kPanel, b_bytes = BN * 128;            // of a plane and stage
    static constexpr int stage = 2 * (a_bytes + b_bytes);
    static constexpr int stages = BN == 256 ? 2 : BN == 128 ? 3 : 4;
    static constexpr int smem = stages * stage + 1024;
    static constexpr int cols = 2 * BN;                                   // of tensor memory
};

__device__ __forceinline__ void sum_warps_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSumWarps * 32) : "memory"); }

template <int BN, Kind K, typename T>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const Product p) {
    using L = Tile<BN>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t s_bars[4 * L::stages + 3];
    __shared__ uint32_t s_tmem;
    __shared__ int s_dead;
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = uniform(smem_u32(smem));
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    // A stage's planes arrive hi first (full) and lo behind (full_lo); B's hi and A's lo are free (empty) before A's hi and B's lo (empty_lo)
    const uint32_t full = smem_u32(s_bars), full_lo = full + 8 * L::stages, empty = full_lo + 8 * L::stages, empty_lo = empty + 8 * L::stages,
                   d_full = empty_lo + 8 * L::stages, d_free = d_full + 8, fin = d_free + 8;
    constexpr bool kSym = K == kGram || K == kSquare;

    // the tile: i 128 rows, j BN columns
    const int splits = K == kGram ? int(cg::this_cluster().num_blocks()) : 1;
    const int part = K == kGram ? int(cg::this_cluster().block_rank()) : 0;
    const int unit = blockIdx.x / splits;
    const int matrix = unit / p.tiles;
    int t = unit - matrix * p.tiles, i, j;
    if (kSym) {
        i = 0;
        for (;; ++i) {
            const int across = i * 128 / BN + (BN < 128 ? 128 / BN : 1);
            if (t < across) break;
            t -= across;
        }
        j = t;
    } else {
        j = t / p.blocks;
        i = t - j * p.blocks;
    }
    const int k0 = int(int64_t(p.k_panels) * part / splits), k1 = int(int64_t(p.k_panels) * (part + 1) / splits), nk = k1 - k0;

    next_may_begin();
    if (threadIdx.x == 0) {
        s_dead = 0;
        for (int s = 0; s < L::stages; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(full_lo + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
            bar_init(empty_lo + 8 * s, 1);
        }
        bar_init(d_full, 1);
        bar_init(d_free, kSumWarps);
        bar_init(fin, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kSumWarps + 1) tmem_alloc(smem_u32(&s_tmem), L::cols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(&s_tmem));
    volatile int* dead = &s_dead;
    unsigned* status = &ortho_status_word;
    wait_for_last();  // its results are read, and what it read is written

    constexpr int kCols = BN / 4;  // of a warp
    float acc[kCols];
    const int quad = warp & 3, quarter = warp >> 2;
    const int row = quad * 32 + lane;  // of the tile
    if (warp < kSumWarps) {
        // ------------------------------------------------------------------------- sums
        const uint32_t from = tmem + uint32_t(quarter * kCols) + (uint32_t(quad * 32) << 16);
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
        bool ok = true;
        for (int r = 0; r < nk && ok; ++r) {  // panel by panel: 64 terms (two cost as much, and cut twice as much)
            ok = warp_wait(d_full, r & 1, dead, status);
            if (!ok) break;
            fence_after();
#pragma unroll
            for (int b = 0; b < kCols / 16; ++b) {
                float v[16];
                tmem_ld16(from + 16 * b, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int c = 0; c < 16; ++c) acc[16 * b + c] = fmaf(v[c], uncut(4), acc[16 * b + c]);
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(d_free);
        }
        if (ok) ok = warp_wait(fin, 0, dead, status);
        if (ok) {
            fence_after();
#pragma unroll
            for (int b = 0; b < kCols / 16; ++b) {
                float v[16];
                tmem_ld16(from + BN + 16 * b, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int c = 0; c < 16; ++c) acc[16 * b + c] = fmaf(v[c], kLoInv, acc[16 * b + c]);
            }
        }
    } else if (warp == kSumWarps) {
        // ------------------------------------------------------------------------ loads
        if (lane == 0) {
            const char* A = p.A + int64_t(matrix) * 2 * p.a_plane + int64_t(i) * p.a_panels * kPanel;
            const char* B = p.B + int64_t(matrix) * 2 * p.b_plane;
            // a tile's last column blocks may lie outside the matrix: their columns are not used
            constexpr int kPart = BN < 128 ? BN * 128 : kPanel;  // bytes of a panel's rows in the tile
            const int b_blocks = !kSym ? 0 : BN < 128 ? 1 : min(BN / 128, p.blocks - j * (BN / 128));
            const uint32_t bytes = L::a_bytes + (kSym ? b_blocks * kPart : L::b_bytes);  // of a plane
            int k = 0;
            for (; k < nk; ++k) {
                const int s = k % L::stages, kp = k0 + k;
                const uint32_t to = sb + uint32_t(s * L::stage), parity = (k / L::stages - 1) & 1;
                auto load_a = [&](int q, uint32_t bar) { bulk_load(to + q * L::a_bytes, A + q * p.a_plane + int64_t(kp) * kPanel, kPanel, bar); };
                auto load_b = [&](int q, uint32_t bar) {
                    const uint32_t tb = to + 2 * L::a_bytes + q * L::b_bytes;
                    if (kSym) {
                        for (int b = 0; b < b_blocks; ++b) {
                            const int first = j * BN + b * 128;  // row of B
                            bulk_load(tb + b * kPart, B + q * p.b_plane + (int64_t(first >> 7) * p.b_panels + kp) * kPanel + (first & 127) * 128,
                                      kPart, bar);
                        }
                    } else {
                        const char* src = B + q * p.b_plane + (int64_t(kp >> 1) * p.b_panels + j * (BN / 64)) * kPanel + (kp & 1) * (kPanel / 2);
#pragma unroll
                        for (int b = 0; b < BN / 64; ++b) bulk_load(tb + b * (kPanel / 2), src + b * kPanel, kPanel / 2, bar);
                    }
                };
                if (k >= L::stages && !bar_wait(empty + 8 * s, parity, dead, status)) break;
                arrive_tx(full + 8 * s, bytes);
                arrive_tx(full_lo + 8 * s, bytes);
                load_b(0, full + 8 * s);
                load_a(1, full_lo + 8 * s);
                if (k >= L::stages) bar_wait_last(empty_lo + 8 * s, parity, status);  // 4 instructions behind: they end
                load_a(0, full + 8 * s);
                load_b(1, full_lo + 8 * s);
            }
            // what was loaded has landed before the block ends, where a wait was given up too
            for (int l = max(0, k - L::stages); l < k; ++l) {
                bar_wait_last(full + 8 * (l % L::stages), (l / L::stages) & 1, status);
                bar_wait_last(full_lo + 8 * (l % L::stages), (l / L::stages) & 1, status);
            }
        }
        __syncwarp();
    } else {
        // --------------------------------------------------------------- matrix instructions
        const uint32_t lead = elect_lane();
        const uint32_t id = mma_desc<__half>(BN, !kSym);
        const uint32_t d_hi = tmem, d_lo = tmem + BN;
        bool ok = true;
        for (int k = 0; k < nk && ok; ++k) {
            const int s = k % L::stages;
            ok = warp_wait(full + 8 * s, (k / L::stages) & 1, dead, status);
            if (ok && k > 0) {
                ok = warp_wait(d_free, (k - 1) & 1, dead, status);
                fence_after();
            }
            if (!ok) break;
            const uint32_t a = own_offset(sb) + uint32_t(s * L::stage), b = a + 2 * L::a_bytes;
            auto da = [&](int plane, int q) { return desc_cols(a + plane * L::a_bytes, q); };
            auto db = [&](int plane, int q) {
                return kSym ? desc_cols(b + plane * L::b_bytes, q) : desc_rows(b + plane * L::b_bytes, q, kPanel / 2);
            };
#pragma unroll
            for (int q = 0; q < 4; ++q) mma_ss(lead, d_hi, da(0, q), db(0, q), id, q > 0);
            mma_commit(lead, d_full);
            ok = warp_wait(full_lo + 8 * s, (k / L::stages) & 1, dead, status);
            if (!ok) break;
#pragma unroll
            for (int q = 0; q < 4; ++q) mma_ss(lead, d_lo, da(1, q), db(0, q), id, k > 0 || q > 0);
            mma_commit(lead, empty + 8 * s);
#pragma unroll
            for (int q = 0; q < 4; ++q) mma_ss(lead, d_lo, da(0, q), db(1, q), id, true);
            mma_commit(lead, empty_lo + 8 * s);
        }
        // every instruction issued has finished before the sums are read to the end and the tensor memory goes
        mma_commit(lead, fin);
        bar_wait_last(fin, 0, status);
        __syncwarp();
    }

    // ------------------------------------------------------------------------------ results
    float* sums = reinterpret_cast<float*>(smem);  // where the stages were: the instructions that read them are done
    if (warp < kSumWarps) {
        if (K == kLast) {
#pragma unroll
            for (int c = 0; c < kCols; ++c) acc[c] *= kHeldInv * kHeldInv * p.scale;
        }
        stage(sums, row, quarter * kCols, BN, acc);
    }
    if (K == kGram && splits > 1) cg::this_cluster().sync();
    if (warp < kSumWarps) {
        sum_warps_sync();
        if (K == kLast) {
            give<T>(sums, kSumWarps * 32, p.side, static_cast<T*>(p.result) + int64_t(matrix) * p.side.matrix, p.vec, i * 128, j * BN, BN);
        } else {
            // a split sum is added up over the cluster: each block takes its share of the columns
            const int share = BN / splits, first = part * share, shift = 31 - __clz(share / 8);
            char* out = p.out + int64_t(matrix) * 2 * p.o_plane;
            // rolled loops: a block runs this once, and unrolled code took longer to fetch than to run
#pragma unroll 1
            for (int t = threadIdx.x; t < 128 << shift; t += kSumWarps * 32) {
                const int r = t >> shift, k = (first >> 3) + (t & ((1 << shift) - 1)), R = i * 128 + r, C = j * BN + 8 * k;
                if (kSym && (C >> 7) > i) continue;  // above the diagonal
                float v[8];
                staged_row(sums, r, k, BN, v);
                if (K == kGram && splits > 1) {
                    staged_row(cg::this_cluster().map_shared_rank(sums, 0), r, k, BN, v);
                    for (int b = 1; b < splits; ++b) {
                        float u[8];
                        staged_row(cg::this_cluster().map_shared_rank(sums, b), r, k, BN, u);
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[q] += u[q];
                    }
                }
                const int64_t at = (int64_t(i) * p.o_panels + (C >> 6)) * kPanel + in_panel(r, C & 63);
                const float f = K == kSquare ? kHeldInv * p.c : kHeldInv;
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] *= f;
                if (K == kSquare && p.b != 0.f) {
                    const Chunk own(p.own + int64_t(matrix) * 2 * p.o_plane + at, p.o_plane);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] = fmaf(p.b, own.value(q), v[q]);
                }
                if (kSym && R < p.m && uint32_t(R - C) < 8u) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (C + q == R) v[q] += p.diagonal * kHeld;
                }
                Chunk(v).store(out + at, p.o_plane);
                if (kSym && (C >> 7) < i) {  // for the block above the diagonal
                    *reinterpret_cast<float4*>(sums + in_stage(r, 2 * k, BN)) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4*>(sums + in_stage(r, 2 * k + 1, BN)) = make_float4(v[4], v[5], v[6], v[7]);
                }
            }
            if (kSym) {
                sum_warps_sync();
                // rows and columns change places
                const int columns = min(share, i * 128 - j * BN - first);  // those of blocks below the diagonal
#pragma unroll 1
                for (int t = threadIdx.x; t < columns * 16; t += kSumWarps * 32) {
                    const int c = first + (t >> 4), k = t & 15, C = j * BN + c;
                    float v[8];
                    staged_column(sums, c, k, BN, v);
                    Chunk(v).store(out + (int64_t(C >> 7) * p.o_panels + 2 * i + (k >> 3)) * kPanel + in_panel(C & 127, (k & 7) * 8), p.o_plane);
                }
            }
        }
    }
    if (K == kGram && splits > 1) cg::this_cluster().sync();  // the others have read this block's sums
    fence_before();
    __syncthreads();
    if (warp == kSumWarps + 1) {
        fence_after();
        tmem_free(tmem, L::cols);
    }
}

// ------------------------------------------------------------------------------------ on chip
//
// A cluster has a matrix, each of its blocks up to 256 of X's columns (4 panels) and all of P.  P's terms are summed over the
// cluster: the blocks' partial sums lie where P will be, each block adds up some rows and writes them to all.

constexpr int kChipThreads = 512, kChipPanels = 4;  // all add up and write; warp 0 issues the matrix instructions, which all wait for
constexpr int kChipSmem = 2 * kChipPanels * kPanel + 4 * kPanel + 1024;
constexpr int kChipBlocks = 8;  // of a cluster at most

struct Chip {
    Side g, out;
    int panels;  // of a block
    int steps;
    float shift, b, c, diagonal, scale;  // a step forms R = P + shift I and M = c R R + b R + diagonal I
    double eps;
    bool vec_in, vec_out;
};

template <typename T>
__global__ void __launch_bounds__(kChipThreads, 1) chip_kernel(const Chip p, const T* gp, T* op) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t s_bar;
    __shared__ uint32_t s_tmem;
    __shared__ int s_dead;
    __shared__ Squares s_norm;
    __shared__ Factor s_factor;
    char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    char* xs = smem + 4 * kPanel;  // P: hi panels 0, 1, lo 0, 1; X: hi panels, lo panels
    const uint32_t sp = own_offset(uniform(smem_u32(smem))), sx = sp + 4 * kPanel;  // for descriptors
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int matrix = blockIdx.x / blocks;
    const T* g = gp + int64_t(matrix) * p.g.matrix;
    T* out = op + int64_t(matrix) * p.out.matrix;
    const int c0 = rank * p.panels * 64, width = p.panels * 64;  // this block's columns
    const int cols = max(0, min(width, p.g.n - c0));             // those inside the matrix
    const uint32_t x_plane = uint32_t(p.panels * kPanel), p_plane = 2 * kPanel;
    const uint32_t bar = smem_u32(&s_bar);
    if (threadIdx.x == 0) {
        s_dead = 0;
        bar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(smem_u32(&s_tmem), 512);

    // X_0.  A thread has 8 columns of a row in each half panel (64 rows of 64 columns): lanes along the values that are consecutive in G
    float v[2 * kChipPanels][8];
    auto place = [&](int u, int& r, int& c) {
        const int t = threadIdx.x;
        r = p.g.turned ? t & 127 : (u & 1) * 64 + (t >> 3);
        c = (u >> 1) * 64 + (p.g.turned ? ((u & 1) * 4 + (t >> 7)) * 8 : (t & 7) * 8);
    };
    Squares squares;
#pragma unroll
    for (int u = 0; u < 2 * kChipPanels; ++u)
        if (u < 2 * p.panels) {
            int r, c;
            place(u, r, c);
            const int left = r < p.g.m ? cols - c : 0;
            if (p.g.turned) {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[u][k] = k < left ? widen(g[(c0 + c + k) * p.g.row + r]) : 0.f;
            } else {
                load_some<T, 8>(g + (left > 0 ? r * p.g.row + c0 + c : 0), left, p.vec_in, v[u]);
            }
        }
#pragma unroll
    for (int u = 0; u < 2 * kChipPanels; ++u)
        if (u < 2 * p.panels) squares.add_all(v[u]);
    fence_before();
    const Squares sum = block_squares<16>(squares);  // (and the tensor memory's address is there)
    fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(&s_tmem));
    if (threadIdx.x == 0) s_norm = sum;
    if (blocks > 1) {
        cluster.sync();
        if (threadIdx.x == 0) {
            Squares total;
            for (int b = 0; b < blocks; ++b) total.add(*cluster.map_shared_rank(&s_norm, b));
            s_factor = Factor(total, p.eps);
        }
    } else if (threadIdx.x == 0) {
        s_factor = Factor(sum, p.eps);
    }
    __syncthreads();
    const Factor inv = s_factor;
#pragma unroll
    for (int u = 0; u < 2 * kChipPanels; ++u)
        if (u < 2 * p.panels) {
            int r, c;
            place(u, r, c);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[u][k] = inv.of(v[u][k]) * kHeld;
            Chunk(v[u]).store(xs + (c >> 6) * kPanel + in_panel(r, c & 63), x_plane);
        }

    volatile int* dead = &s_dead;
    unsigned* status = &ortho_status_word;
    const int quad = warp & 3, quarter = warp >> 2, row = quad * 32 + lane;
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    const uint32_t lead = warp == 0 ? elect_lane() : 0;
    const int k16 = (p.g.m + 15) / 16;            // instructions of a sum over the rows
    const int c16 = max(1, (cols + 15) / 16);     // and over this block's columns; one at least: zeros
    const int m16 = 16 * k16;                     // P's rows and columns in use; what lies beyond is read by no sum that counts
    const bool rows_live = quad * 32 < p.g.m, p_live = rows_live && quarter * 32 < m16;
    const uint32_t id_p = mma_desc<__half>(m16, false), id_x = mma_desc<__half>(width, true);
    const bool wide = width > 128;
    uint32_t phase = 0;
    bool ok = true;
    // all writes of operands are done; the instructions that `issue` forms run, and everyone waits for them
    auto product = [&](auto issue) {
        fence_async();
        fence_before();
        ok = __syncthreads_and(ok);  // after a wait that was given up the block goes on to the end, for the others' sake
        if (!ok) return;
        if (warp == 0) {
            fence_after();
            issue();
            mma_commit(lead, bar);
        }
        ok = warp_wait(bar, phase, dead, status);
        phase ^= 1;
        fence_after();
    };
    // Accumulators of a product of up to 128 columns: lo at column 256, hi hi in turn at 0, 128 and 384, so that each cuts a third of
    // the sum a third as often; a wider product has one, and lo at 256.
    auto hi_at = [&](int k) { return tmem + (k % 3 == 2 ? 384u : uint32_t(k % 3) * 128u); };
    // columns c .. c + 31 of a product of n instructions, as pairs
    auto sums = [&](int c, int n, bool one, float (&v)[32]) {
        float u[32];
        const uint32_t at = uint32_t(c) + lanes;
        tmem_ld32(tmem + at, v);
        tmem_ld32(tmem + 256 + at, u);
        tmem_wait_ld(v);
        tmem_wait_ld(u);
        const float f0 = uncut(one ? n : (n + 2) / 3) * kHeldInv, lo = kLoInv * kHeldInv;
        F2 w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = fma2(F2(v[2 * i], v[2 * i + 1]), F2(f0, f0), F2(u[2 * i], u[2 * i + 1]) * F2(lo, lo));
        if (!one)
            for (int a = 1; a < min(n, 3); ++a) {
                tmem_ld32(hi_at(a) + at, u);
                tmem_wait_ld(u);
                const float f = uncut((n + 2 - a) / 3) * kHeldInv;
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = fma2(F2(u[2 * i], u[2 * i + 1]), F2(f, f), w[i]);
            }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 b = w[i].both();
            v[2 * i] = b.x, v[2 * i + 1] = b.y;
        }
    };
    auto on_diagonal = [&](int c, float d, float (&v)[32]) {  // columns c .. c + 31
        if (row < p.g.m && uint32_t(row - c) < 32u) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i == row) v[i] += d * kHeld;
        }
    };
    for (int step = 0; step < p.steps; ++step) {
        // R = X X^T + shift I
        product([&] {
            for (int k = 0; k < c16; ++k) {
                const uint32_t x = sx + uint32_t(k >> 2) * kPanel;
                const uint64_t h = desc_cols(x, k & 3), l = desc_cols(x + x_plane, k & 3);
                mma_ss(lead, hi_at(k), h, h, id_p, k > 2);
                mma_ss(lead, tmem + 256, h, l, id_p, k > 0);
                mma_ss(lead, tmem + 256, l, h, id_p, true);
            }
        });
        if (blocks == 1) {
            if (p_live) {
                const int c = quarter * 32;
                float v[32];
                sums(c, c16, false, v);
                on_diagonal(c, p.shift, v);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    Chunk(v + 8 * k).store(smem + (c >> 6) * kPanel + in_panel(row, (c & 63) + 8 * k), p_plane);
            }
        } else {
            float* part = reinterpret_cast<float*>(smem);  // [128][128], 16-byte chunks of a row exchanged by its number
            auto at = [](int r, int chunk) { return r * 128 + ((chunk ^ (r & 31)) << 2); };
            if (p_live) {
                const int c = quarter * 32;
                float v[32];
                sums(c, c16, false, v);
                if (rank == 0) on_diagonal(c, p.shift, v);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<float4*>(part + at(row, c / 4 + k)) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
            cluster.sync();
            // each block adds up its share of the rows: 8 columns a thread, two times for two blocks of all 128 rows
            const int chunks = m16 / 8, share = (m16 + blocks - 1) / blocks;
            auto exchange = [&](auto count) {
                constexpr int B = decltype(count)::value, U = B == 2 ? 2 : 1;
                float v[U][8];
                int r[U], c[U];
                bool on[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int t = threadIdx.x + u * kChipThreads, row_of = t / chunks;
                    r[u] = rank * share + row_of, c[u] = (t - row_of * chunks) * 8;
                    on[u] = row_of < share && r[u] < m16;
                    if (on[u]) {
                        float4 x[B], y[B];
#pragma unroll
                        for (int b = 0; b < B; ++b) {
                            const float* other = cluster.map_shared_rank(part, b);
                            x[b] = *reinterpret_cast<const float4*>(other + at(r[u], c[u] / 4));
                            y[b] = *reinterpret_cast<const float4*>(other + at(r[u], c[u] / 4 + 1));
                        }
#pragma unroll
                        for (int q = 0; q < 8; ++q) v[u][q] = 0.f;
#pragma unroll
                        for (int b = 0; b < B; ++b) {
                            v[u][0] += x[b].x, v[u][1] += x[b].y, v[u][2] += x[b].z, v[u][3] += x[b].w;
                            v[u][4] += y[b].x, v[u][5] += y[b].y, v[u][6] += y[b].z, v[u][7] += y[b].w;
                        }
                    }
                }
                cluster.sync();
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (on[u]) {
                        const Chunk w(v[u]);
#pragma unroll
                        for (int b = 0; b < B; ++b)
                            w.store(cluster.map_shared_rank(smem, b) + (c[u] >> 6) * kPanel + in_panel(r[u], c[u] & 63), p_plane);
                    }
            };
            if (blocks == 2) exchange(std::integral_constant<int, 2>());
            else if (blocks == 4) exchange(std::integral_constant<int, 4>());
            else exchange(std::integral_constant<int, 8>());
            fence_async_all();
            cluster.sync();
        }
        // M = c R R + b R + diagonal I, where R was
        product([&] {
            for (int k = 0; k < k16; ++k) {
                const uint32_t x = sp + uint32_t(k >> 2) * kPanel;
                const uint64_t h = desc_cols(x, k & 3), l = desc_cols(x + p_plane, k & 3);
                mma_ss(lead, hi_at(k), h, h, id_p, k > 2);
                mma_ss(lead, tmem + 256, h, l, id_p, k > 0);
                mma_ss(lead, tmem + 256, l, h, id_p, true);
            }
        });
        if (p_live) {
            const int c = quarter * 32;
            float v[32];
            sums(c, k16, false, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= p.c;
            on_diagonal(c, p.diagonal, v);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                char* to = smem + (c >> 6) * kPanel + in_panel(row, (c & 63) + 8 * k);
                if (p.b != 0.f) {
                    const Chunk own(to, p_plane);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[8 * k + q] = fmaf(p.b, own.value(q), v[8 * k + q]);
                }
                Chunk(v + 8 * k).store(to, p_plane);
            }
        }
        // X = M X
        product([&] {
            for (int k = 0; k < k16; ++k) {
                const uint32_t m = sp + uint32_t(k >> 2) * kPanel;
                const uint64_t mh = desc_cols(m, k & 3), ml = desc_cols(m + p_plane, k & 3);
                const uint64_t xh = desc_rows(sx, k), xl = desc_rows(sx + x_plane, k);
                mma_ss(lead, wide ? tmem : hi_at(k), mh, xh, id_x, k > (wide ? 0 : 2));
                mma_ss(lead, tmem + 256, mh, xl, id_x, k > 0);
                mma_ss(lead, tmem + 256, ml, xh, id_x, true);
            }
        });
        const bool last = step + 1 == p.steps;
        if (rows_live)
            for (int b = quarter; b < p.panels * 2; b += 4) {
                float v[32];
                sums(32 * b, k16, wide, v);
                if (!last) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        Chunk(v + 8 * k).store(xs + (b >> 1) * kPanel + in_panel(row, (b & 1) * 32 + 8 * k), x_plane);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] *= kHeldInv * p.scale;
                    stage(reinterpret_cast<float*>(xs), row, 32 * b, width, v);
                }
            }
        if (last) {
            __syncthreads();
            give<T>(reinterpret_cast<const float*>(xs), kChipThreads, p.out, out, p.vec_out, 0, c0, width);
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 0) {
        if (!ok) bar_wait_last(bar, phase ^ 1, status);
        __syncwarp();
        fence_after();
        tmem_free(tmem, 512);
    }
}

// ----------------------------------------------------------------------------------------- host

int up(int v, int to) { return (v + to - 1) / to * to; }

struct Sizes {
    int m, n, blocks, x_panels, p_panels;  // panels of a row block
    size_t x_plane, p_plane;
    bool turned, fits, chip;  // fits: on chip; chip: runs there
    int chip_blocks, chip_panels;
};
Sizes sizes_of(const OrthoShape& s) {
    Sizes z;
    z.turned = s.rows > s.cols;
    z.m = std::min(s.rows, s.cols), z.n = std::max(s.rows, s.cols);
    z.blocks = up(z.m, 128) / 128;
    z.x_panels = up(z.n, 256) / 64;
    z.p_panels = 2 * z.blocks;
    z.x_plane = size_t(z.blocks) * z.x_panels * kPanel;
    z.p_plane = size_t(z.blocks) * z.p_panels * kPanel;
    const int panels = up(z.n, 64) / 64;
    z.chip_blocks = 1;
    while (z.chip_blocks < kChipBlocks && panels > z.chip_blocks * kChipPanels) z.chip_blocks *= 2;
    // Of the largest clusters the card holds some 9 at once (they do not span its groups of SMs): 16 matrices of 128 x 2000 took 176 us in
    // two rounds, 122 us in tiles, and 8 took 90 against 148.
    z.fits = z.m <= 128 && z.n <= 64 * kChipPanels * kChipBlocks && (z.chip_blocks < kChipBlocks || s.n_matrices <= 9);
    z.chip = z.fits && s.steps > 0;
    z.chip_panels = (panels + z.chip_blocks - 1) / z.chip_blocks;
    return z;
}

struct Parts {
    Squares* norm;
    char *x[2], *p, *q;
    size_t bytes;
};
Parts parts_of(const OrthoShape& s, const Sizes& z, void* ws) {
    char* at = static_cast<char*>(ws);
    size_t used = 0;
    auto take = [&](size_t bytes) {
        char* r = at + used;
        used += align256(bytes);
        return r;
    };
    const size_t b = s.n_matrices;
    Parts p = {};
    // the same whatever the number of steps
    p.norm = reinterpret_cast<Squares*>(take(b * kNormBlocks * sizeof(Squares)));
    if (!z.fits) {
        p.x[0] = take(b * 2 * z.x_plane);
        p.x[1] = take(b * 2 * z.x_plane);
        p.p = take(b * 2 * z.p_plane);
        p.q = take(b * 2 * z.p_plane);
    }
    p.bytes = used;
    return p;
}

// follows: the kernel waits for the launch before it itself.
template <typename... P, typename... Q>
cudaError_t launch(void (*k)(P...), int64_t blocks, int threads, int cluster, bool follows, size_t smem, cudaStream_t st, Q... args) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(unsigned(blocks));
    c.blockDim = dim3(unsigned(threads));
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = unsigned(cluster);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = follows ? 2 : 1;
    return cudaLaunchKernelEx(&c, k, static_cast<P>(args)...);
}

int sym_tiles(int blocks, int bn) {
    int t = 0;
    for (int i = 0; i < blocks; ++i) t += i * 128 / bn + (bn < 128 ? 128 / bn : 1);
    return t;
}

// One product of every matrix (T: the type of kLast's result).  Tiles of 256 columns where they fill the card, since they read the least;
// smaller ones where only they give every SM one: what follows the sums takes a block's threads as long as they do, for products of
// 256 x 256 (25 of them, five steps: 117 us with tiles of 128, 99 with 64).
template <int BN, Kind K, typename T>
cudaError_t product(const Product& p, int64_t tiles, int sms, cudaStream_t st) {
    int splits = 1;  // of a long sum, where there are few tiles
    if (K == kGram)
        while (splits < kMaxSplits && splits * 8 < BN && tiles * splits * 2 <= sms && p.k_panels >= splits * 2 * 4) splits *= 2;
    return launch(product_kernel<BN, K, T>, tiles * splits, kThreads, splits, true, Tile<BN>::smem, st, p);
}
template <Kind K, typename T>
cudaError_t product(Product p, int matrices, int columns, int sms, cudaStream_t st) {
    constexpr bool kSym = K == kGram || K == kSquare;
    auto tiles = [&](int bn) { return p.tiles = kSym ? sym_tiles(p.blocks, bn) : p.blocks * (up(columns, bn) / bn), int64_t(p.tiles) * matrices; };
    if (tiles(256) >= sms * 3 / 4) return product<256, K, T>(p, tiles(256), sms, st);
    if (tiles(64) <= sms) return product<64, K, T>(p, tiles(64), sms, st);
    return product<128, K, T>(p, tiles(128), sms, st);
}

template <typename T>
cudaError_t run(const OrthoShape& s, const void* gp, void* op, void* ws, int sms, cudaStream_t st) {
    const Sizes z = sizes_of(s);
    const Parts w = parts_of(s, z, ws);
    const T* g = static_cast<const T*>(gp);
    T* out = static_cast<T*>(op);
    const Side in = {z.m, z.n, z.turned, s.g_matrix, s.g_row}, to = {z.m, z.n, z.turned, s.o_matrix, s.o_row};
    auto aligned = [](const void* t, int64_t row, int64_t matrix) {
        return ((reinterpret_cast<uintptr_t>(t) | uintptr_t(row) * sizeof(T) | uintptr_t(matrix) * sizeof(T)) & 15u) == 0;
    };
    const bool vec_in = aligned(gp, s.g_row, s.g_matrix), vec_out = aligned(op, s.o_row, s.o_matrix);
    // a I + b P + c P P = c R R + (a - b^2 / 4c) I with R = P + b / 2c I: near the end, where P is near I, R is small, and so
    // are its products' errors.  Where b / 2c is not of P's size the sum is formed as it stands.
    const double half = s.c != 0 ? s.b / (2 * s.c) : 0.0;
    const bool whole = s.c != 0 && std::fabs(half) <= 2.0;
    const float shift = whole ? float(half) : 0.f, b = whole ? 0.f : float(s.b);
    const float diagonal = float(whole ? s.a - s.b * half / 2 : s.a);
    if (z.chip) {
        const Chip c = {in, to, z.chip_panels, s.steps, shift, b, float(s.c), diagonal, float(s.scale), s.eps, vec_in, vec_out};
        return launch(chip_kernel<T>, int64_t(s.n_matrices) * z.chip_blocks, kChipThreads, z.chip_blocks, false, kChipSmem, st, c, g, out);
    }
    const int parts = int(std::min<int64_t>(kNormBlocks, (int64_t(s.rows) * ((s.cols + 7) / 8) + 1023) / 1024));
    norm_kernel<T><<<dim3(parts, s.n_matrices), 256, 0, st>>>(s.rows, s.cols, s.g_matrix, s.g_row, vec_in, g, w.norm);
    if (s.steps == 0) {
        scale_kernel<T><<<dim3(std::min(s.rows, 1024), s.n_matrices), 256, 0, st>>>(s.rows, s.cols, s.g_matrix, s.g_row, s.o_matrix, s.o_row,
                                                                                   float(s.scale), g, w.norm, parts, s.eps, out);
        return cudaGetLastError();
    }
    take_kernel<T><<<dim3(z.x_panels, z.blocks * 2, s.n_matrices), 256, 0, st>>>(in, vec_in, g, w.norm, parts, s.eps, z.x_panels, z.x_plane,
                                                                                 w.x[0]);
    cudaError_t e = cudaGetLastError();
    for (int i = 0; i < s.steps && e == cudaSuccess; ++i) {
        const char* x = w.x[i & 1];
        Product p = {};
        p.blocks = z.blocks, p.m = z.m;
        p.A = p.B = x, p.a_plane = p.b_plane = z.x_plane, p.a_panels = p.b_panels = z.x_panels;
        p.out = w.p, p.o_plane = z.p_plane, p.o_panels = z.p_panels;
        p.k_panels = up(z.n, 64) / 64, p.diagonal = shift;
        e = product<kGram, float>(p, s.n_matrices, z.m, sms, st);
        if (e != cudaSuccess) break;
        p.A = p.B = p.own = w.p, p.a_plane = p.b_plane = z.p_plane, p.a_panels = p.b_panels = z.p_panels;
        p.out = w.q;
        p.k_panels = up(z.m, 64) / 64, p.diagonal = diagonal, p.b = b, p.c = float(s.c);
        e = product<kSquare, float>(p, s.n_matrices, z.m, sms, st);
        if (e != cudaSuccess) break;
        p.A = w.q, p.B = x, p.b_plane = z.x_plane, p.b_panels = z.x_panels;
        p.out = w.x[(i + 1) & 1], p.o_plane = z.x_plane, p.o_panels = z.x_panels;
        p.side = to, p.scale = float(s.scale), p.vec = vec_out, p.result = out;
        e = i + 1 < s.steps ? product<kApply, float>(p, s.n_matrices, z.n, sms, st) : product<kLast, T>(p, s.n_matrices, z.n, sms, st);
    }
    return e;
}

}  // namespace

size_t ortho_workspace(const OrthoShape& s) { return s.n_matrices == 0 ? 0 : parts_of(s, sizes_of(s), nullptr).bytes; }

cudaError_t launch_ortho(const OrthoShape& s, const void* g, void* out, void* ws, int sms, cudaStream_t st) {
    switch (s.dtype) {
        case UVU_F32: return run<float>(s, g, out, ws, sms, st);
        case UVU_BF16: return run<__nv_bfloat16>(s, g, out, ws, sms, st);
        case UVU_F16: return run<__half>(s, g, out, ws, sms, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t ortho_status(unsigned* word, bool reset) {
    cudaError_t e = cudaMemcpyFromSymbol(word, ortho_status_word, sizeof(unsigned));
    if (e != cudaSuccess || !reset) return e;
    const unsigned z = 0;
    return cudaMemcpyToSymbol(ortho_status_word, &z, sizeof(unsigned));
}

}  // namespace uvu
