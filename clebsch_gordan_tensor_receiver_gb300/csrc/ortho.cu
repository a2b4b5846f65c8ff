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
// those of large matrices (1 / sqrt(m n)) normal numbers of fp16 and those near 1 far from its largest.
//
// An accumulating matrix instruction (16 terms) cuts its sum towards zero, by 2^-24 of it in the mean (measured: 2.8 2^-24 after
// four of them, 7.7 after eight, on sums of one sign).  So the hi hi accumulator is taken into fp32 registers every 128 terms, while the
// lo products, two thirds of the instructions, run, and the mean of what was cut is put back: a factor 1 + 2^-24 for each instruction.
// Without it five steps on 64 x 1664 values were off by 2.4e-6, the plain form in fp32 by 9.6e-7.
//
// A matrix is kept in panels of 128 rows and 64 columns, 16 KB each, whose bytes lie as the matrix instruction reads them
// (128-byte swizzle): a panel is loaded by one bulk copy, and no tensor map is needed.
//
// Two forms.  On chip, for m <= 128 and n <= 2048: a block, or a cluster of up to 8 that splits the columns, keeps X and P in shared
// memory from the first step to the last; one launch.  Else a kernel for each product, of 128 x 256 or 128 x 128 tiles.
#include <cooperative_groups.h>

#include <algorithm>
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
// Ordinary writes, of this block's shared memory or another's, come before asynchronous reads.
__device__ __forceinline__ void fence_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// hi in the low half, lo in the high one.
__device__ __forceinline__ uint32_t split(float v) {
    const __half hi = __float2half_rn(v);
    const __half lo = __float2half_rn((v - __half2float(hi)) * kLo);
    return uint32_t(__half_as_ushort(hi)) | uint32_t(__half_as_ushort(lo)) << 16;
}
__device__ __forceinline__ float joined(uint32_t hi, uint32_t lo) {
    return fmaf(__half2float(__ushort_as_half(uint16_t(lo))), kLoInv, __half2float(__ushort_as_half(uint16_t(hi))));
}
// Eight values' halves as the 16 bytes of each plane.
__device__ __forceinline__ void planes_of(const uint32_t (&w)[8], uint4& hi, uint4& lo) {
    hi = make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410), __byte_perm(w[4], w[5], 0x5410),
                    __byte_perm(w[6], w[7], 0x5410));
    lo = make_uint4(__byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632), __byte_perm(w[4], w[5], 0x7632),
                    __byte_perm(w[6], w[7], 0x7632));
}
// A shared-memory address for an operand's descriptor, which has room for the offset in the block's own memory alone: in a cluster the
// address also has the block's rank, in its upper byte.
__device__ __forceinline__ uint32_t own_offset(uint32_t address) { return address & 0x3FFFFu; }
// Where a panel holds row r (of its 128) and column c (of its 64).
__device__ __forceinline__ uint32_t in_panel(int r, int c) {
    return uint32_t((r >> 3) * 1024 + (r & 7) * 128 + ((((c >> 3) ^ r) & 7) << 4) + (c & 7) * 2);
}

// A squared norm in fp32 whatever the values' size: the squares of large and of small ones are summed at scales of their own.
struct Squares {
    float small = 0.f, mid = 0.f, large = 0.f;
    __device__ __forceinline__ void add(float v) {
        v = fabsf(v);
        if (v > 0x1p50f) {
            v *= 0x1p-60f;
            large = fmaf(v, v, large);
        } else if (v < 0x1p-50f) {
            v *= 0x1p60f;
            small = fmaf(v, v, small);
        } else {
            mid = fmaf(v, v, mid);  // a NaN comes here
        }
    }
    __device__ __forceinline__ double total() const { return double(small) * 0x1p-120 + double(mid) + double(large) * 0x1p120; }
};
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// X's element (r, c) in G: G[r][c], or G[c][r] where G is turned.
struct Side {
    int m, n;
    bool turned;
    int64_t matrix, row;
    __device__ __forceinline__ int64_t at(int r, int c) const { return turned ? c * row + r : r * row + c; }
};

// ------------------------------------------------------------------------------- norm and planes

constexpr int kNormBlocks = 64;  // partial sums of a matrix at most

template <typename T>
__global__ void __launch_bounds__(512) norm_kernel(int rows, int cols, int64_t g_matrix, int64_t g_row, const T* g, double* part) {
    const T* a = g + int64_t(blockIdx.y) * g_matrix;
    Squares s;
    for (int r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < cols; c += blockDim.x) s.add(widen(a[r * g_row + c]));
    __shared__ double s_sum[16];
    const double v = warp_sum(s.total());
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0;
        for (int w = 0; w < 16; ++w) t += s_sum[w];
        part[blockIdx.y * kNormBlocks + blockIdx.x] = t;
    }
}

// The factor 1 / (|G| + eps), as two: fp32 does not hold the inverse of the smallest norms.  Zeros stay zeros, with eps = 0 too; an
// infinity makes the whole matrix NaN, as a NaN does.
struct Factor {
    float first, second;
    __device__ __forceinline__ Factor() {}
    __device__ __forceinline__ Factor(double squares, double eps) {
        const double inv = squares == 0.0 ? 0.0 : isinf(squares) ? double(NAN) : 1.0 / (sqrt(squares) + eps);
        first = inv > 0x1p100 ? 0x1p60f : 1.f;
        second = float(inv / double(first));
    }
    __device__ __forceinline__ float of(float v) const { return v * first * second; }
};

// That of the block's matrix, in every thread of the block.
__device__ __forceinline__ Factor inverse_norm(const double* part, int parts, double eps) {
    __shared__ Factor s_inv;
    if (threadIdx.x < 32) {
        double v = 0;
        for (int i = threadIdx.x; i < parts; i += 32) v += part[i];
        v = warp_sum(v);
        if (threadIdx.x == 0) s_inv = Factor(v, eps);
    }
    __syncthreads();
    return s_inv;
}

// X_0's planes, a 64 x 64 piece a block: (column panel, half a row block, matrix).
template <typename T>
__global__ void __launch_bounds__(256) take_kernel(Side s, const T* g, const double* part, int parts, double eps, int panels, size_t plane,
                                                   char* x) {
    __shared__ float tile[64][65];
    const Factor inv = inverse_norm(part + int64_t(blockIdx.z) * kNormBlocks, parts, eps);
    const T* a = g + int64_t(blockIdx.z) * s.matrix;
    const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
    for (int i = threadIdx.x; i < 4096; i += 256) {
        const int u = i >> 6, v = i & 63;  // lanes along the values that are consecutive in G
        const int r = r0 + (s.turned ? v : u), c = c0 + (s.turned ? u : v);
        tile[r - r0][c - c0] = r < s.m && c < s.n ? inv.of(widen(a[s.at(r, c)])) * kHeld : 0.f;
    }
    __syncthreads();
    char* to = x + int64_t(blockIdx.z) * 2 * plane + (int64_t(blockIdx.y >> 1) * panels + blockIdx.x) * kPanel;
    for (int i = threadIdx.x; i < 512; i += 256) {
        const int r = i >> 3, c = (i & 7) * 8;
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = split(tile[r][c + k]);
        uint4 hi, lo;
        planes_of(w, hi, lo);
        const uint32_t at = in_panel((blockIdx.y & 1) * 64 + r, c);
        *reinterpret_cast<uint4*>(to + at) = hi;
        *reinterpret_cast<uint4*>(to + plane + at) = lo;
    }
}

// No steps: out = scale X_0.
template <typename T>
__global__ void __launch_bounds__(256) scale_kernel(int rows, int cols, int64_t g_matrix, int64_t g_row, int64_t o_matrix, int64_t o_row,
                                                    float scale, const T* g, const double* part, int parts, double eps, T* out) {
    const Factor inv = inverse_norm(part + int64_t(blockIdx.y) * kNormBlocks, parts, eps);
    const T* a = g + int64_t(blockIdx.y) * g_matrix;
    T* o = out + int64_t(blockIdx.y) * o_matrix;
    for (int r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < cols; c += blockDim.x) o[r * o_row + c] = narrow<T>(inv.of(widen(a[r * g_row + c])) * scale);
}

// Eight results of row r, columns c .. c + 7 of X, to the caller's matrix.
template <typename T>
__device__ __forceinline__ void give(const Side& s, T* out, bool vec, int r, int c, const float (&v)[8]) {
    if (r >= s.m) return;
    if (!s.turned && vec && c + 8 <= s.n) {
        T* o = out + r * s.row + c;
        T t[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = narrow<T>(v[i]);
#pragma unroll
        for (int i = 0; i < int(sizeof(t) / 16); ++i) {
            uint4 q;
            __builtin_memcpy(&q, reinterpret_cast<const char*>(t) + 16 * i, 16);
            reinterpret_cast<uint4*>(o)[i] = q;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < s.n) out[s.at(r, c + i)] = narrow<T>(v[i]);
    }
}

// ------------------------------------------------------------------------------------ one product

enum Kind { kGram, kSquare, kApply, kLast };

struct Product {
    const char *A, *B, *own;  // panels of 128 rows (B of kApply: the rows are the summed index); own: P of kSquare
    char* out;
    size_t a_plane, b_plane, o_plane;      // bytes of a plane; a matrix has two
    int a_panels, b_panels, o_panels;      // of a row block
    int blocks;                            // row blocks of the result
    int k_panels;                          // of 64 summed values
    int tiles;                             // of a matrix
    int m;
    float a, b, c;
    // kLast
    Side side;
    float scale;
    bool vec;
    void* result;
};

constexpr int kThreads = 320;  // 8 warps that add up and write, one that loads, one that issues the matrix instructions
constexpr int kRunPanels = 1;  // panels of 64 terms between two readings of the hi hi accumulator

template <int BN>
struct Tile {
    static constexpr int a_bytes = kPanel, b_bytes = BN * 128;            // of a plane and stage
    static constexpr int stage = 2 * (a_bytes + b_bytes);
    static constexpr int stages = BN == 256 ? 2 : 3;
    static constexpr int smem = stages * stage + 1024;
    static constexpr int cols = BN == 256 ? 512 : 256;                    // of tensor memory
};

template <int BN, Kind K, typename T>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const Product p) {
    using L = Tile<BN>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t s_bars[2 * L::stages + 3];
    __shared__ uint32_t s_tmem;
    __shared__ int s_dead;
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = uniform(smem_u32(smem));
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t full = smem_u32(s_bars), empty = full + 8 * L::stages, d_full = empty + 8 * L::stages, d_free = d_full + 8, fin = d_free + 8;
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
            const int across = i / (BN / 128) + 1;
            if (t < across) break;
            t -= across;
        }
        j = t;
    } else {
        j = t / p.blocks;
        i = t - j * p.blocks;
    }
    const int k0 = int(int64_t(p.k_panels) * part / splits), k1 = int(int64_t(p.k_panels) * (part + 1) / splits), nk = k1 - k0;
    const int runs = (nk + kRunPanels - 1) / kRunPanels;

    if (threadIdx.x == 0) {
        s_dead = 0;
        for (int s = 0; s < L::stages; ++s) {
            bar_init(full + 8 * s, 1);
            bar_init(empty + 8 * s, 1);
        }
        bar_init(d_full, 1);
        bar_init(d_free, 8);
        bar_init(fin, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) tmem_alloc(smem_u32(&s_tmem), L::cols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(&s_tmem));
    volatile int* dead = &s_dead;
    unsigned* status = &ortho_status_word;

    float acc[BN / 2];
    const int quad = warp & 3, half = (warp >> 2) & 1;
    const int row = quad * 32 + lane;  // of the tile
    if (warp < 8) {
        // ------------------------------------------------------------------------- sums
        const uint32_t from = tmem + uint32_t(half * (BN / 2)) + (uint32_t(quad * 32) << 16);
#pragma unroll
        for (int c = 0; c < BN / 2; ++c) acc[c] = 0.f;
        bool ok = true;
        for (int r = 0; r < runs && ok; ++r) {
            ok = warp_wait(d_full, r & 1, dead, status);
            if (!ok) break;
            fence_after();
            const float f = uncut(4 * min(kRunPanels, nk - r * kRunPanels));
#pragma unroll
            for (int b = 0; b < BN / 64; ++b) {
                float v[32];
                tmem_ld32(from + 32 * b, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[32 * b + c] = fmaf(v[c], f, acc[32 * b + c]);
            }
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(d_free);
        }
        if (ok) ok = warp_wait(fin, 0, dead, status);
        if (ok) {
            fence_after();
#pragma unroll
            for (int b = 0; b < BN / 64; ++b) {
                float v[32];
                tmem_ld32(from + BN + 32 * b, v);
                tmem_wait_ld(v);
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[32 * b + c] = fmaf(v[c], kLoInv, acc[32 * b + c]);
            }
        }
    } else if (warp == 8) {
        // ------------------------------------------------------------------------ loads
        if (lane == 0) {
            const char* A = p.A + int64_t(matrix) * 2 * p.a_plane + int64_t(i) * p.a_panels * kPanel;
            const char* B = p.B + int64_t(matrix) * 2 * p.b_plane;
            // a tile's last column blocks may lie outside the matrix: their columns are not used
            const int b_blocks = kSym ? min(BN / 128, p.blocks - j * (BN / 128)) : 0;
            const uint32_t bytes = 2 * (L::a_bytes + (kSym ? b_blocks * kPanel : L::b_bytes));
            int k = 0;
            for (; k < nk; ++k) {
                const int s = k % L::stages;
                if (k >= L::stages && !bar_wait(empty + 8 * s, (k / L::stages - 1) & 1, dead, status)) break;
                const uint32_t to = sb + uint32_t(s * L::stage), bar = full + 8 * s;
                arrive_tx(bar, bytes);
                const int kp = k0 + k;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    bulk_load(to + q * L::a_bytes, A + q * p.a_plane + int64_t(kp) * kPanel, kPanel, bar);
                    const uint32_t tb = to + 2 * L::a_bytes + q * L::b_bytes;
                    if (kSym) {
                        for (int b = 0; b < b_blocks; ++b)
                            bulk_load(tb + b * kPanel, B + q * p.b_plane + (int64_t(j * (BN / 128) + b) * p.b_panels + kp) * kPanel, kPanel, bar);
                    } else {
                        const char* src = B + q * p.b_plane + (int64_t(kp >> 1) * p.b_panels + j * (BN / 64)) * kPanel + (kp & 1) * (kPanel / 2);
#pragma unroll
                        for (int b = 0; b < BN / 64; ++b) bulk_load(tb + b * (kPanel / 2), src + b * kPanel, kPanel / 2, bar);
                    }
                }
            }
            // what was loaded has landed before the block ends, where a wait was given up too
            for (int l = max(0, k - L::stages); l < k; ++l) bar_wait_last(full + 8 * (l % L::stages), (l / L::stages) & 1, status);
        }
        __syncwarp();
    } else {
        // --------------------------------------------------------------- matrix instructions
        const uint32_t lead = elect_lane();
        const uint32_t id = mma_desc<__half>(BN, !kSym);
        const uint32_t d_hi = tmem, d_lo = tmem + BN;
        bool ok = true;
        for (int k = 0; k < nk && ok; ++k) {
            const int s = k % L::stages, r = k / kRunPanels;
            const bool first = k % kRunPanels == 0, last = k % kRunPanels == kRunPanels - 1 || k == nk - 1;
            ok = warp_wait(full + 8 * s, (k / L::stages) & 1, dead, status);
            if (ok && first && r > 0) {
                ok = warp_wait(d_free, (r - 1) & 1, dead, status);
                fence_after();
            }
            if (!ok) break;
            const uint32_t a = own_offset(sb) + uint32_t(s * L::stage), b = a + 2 * L::a_bytes;
            auto da = [&](int plane, int q) { return desc_cols(a + plane * L::a_bytes, q); };
            auto db = [&](int plane, int q) {
                return kSym ? desc_cols(b + plane * L::b_bytes, q) : desc_rows(b + plane * L::b_bytes, q, kPanel / 2);
            };
#pragma unroll
            for (int q = 0; q < 4; ++q) mma_ss(lead, d_hi, da(0, q), db(0, q), id, !first || q > 0);
            if (last) mma_commit(lead, d_full);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                mma_ss(lead, d_lo, da(0, q), db(1, q), id, k > 0 || q > 0);
                mma_ss(lead, d_lo, da(1, q), db(0, q), id, true);
            }
            mma_commit(lead, empty + 8 * s);
        }
        // every instruction issued has finished before the sums are read to the end and the tensor memory goes
        mma_commit(lead, fin);
        bar_wait_last(fin, 0, status);
        __syncwarp();
    }

    // a split sum is added up over the cluster: each block takes its share of the columns
    int c0 = half * (BN / 2), count = BN / 2;  // of the tile; this thread's
    if (K == kGram && splits > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        float* mine = reinterpret_cast<float*>(smem);
        __syncthreads();  // the stages have been read
        if (warp < 8) {
#pragma unroll
            for (int c = 0; c < BN / 2; ++c) mine[(c0 + c) * 128 + row] = acc[c];
        }
        cluster.sync();
        if (warp < 8) {
            count = BN / 2 / splits;
            c0 = part * (BN / splits) + half * count;
#pragma unroll
            for (int c = 0; c < BN / 4; ++c) acc[c] = 0.f;
            for (int s = 0; s < splits; ++s) {
                const float* other = cluster.map_shared_rank(mine, s);
#pragma unroll
                for (int c = 0; c < BN / 4; ++c)
                    if (c < count) acc[c] += other[(c0 + c) * 128 + row];
            }
        }
        cluster.sync();
    }

    if (warp < 8) {
        // ----------------------------------------------------------------------- results
        const int R = i * 128 + row;
        if (K == kLast) {
            T* out = static_cast<T*>(p.result) + int64_t(matrix) * p.side.matrix;
            const float f = kHeldInv * kHeldInv * p.scale;
#pragma unroll
            for (int k = 0; k < BN / 16; ++k) {
                float v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = acc[8 * k + q] * f;
                give<T>(p.side, out, p.vec, R, j * BN + c0 + 8 * k, v);
            }
        } else {
            char* out = p.out + int64_t(matrix) * 2 * p.o_plane;
            const char* own = K == kSquare ? p.own + int64_t(matrix) * 2 * p.o_plane : nullptr;
#pragma unroll
            for (int k = 0; k < BN / 16; ++k) {
                const int C = j * BN + c0 + 8 * k;
                if (8 * k < count && !(kSym && (C >> 7) > i)) {
                    const int64_t at = (int64_t(i) * p.o_panels + (C >> 6)) * kPanel + in_panel(row, C & 63);
                    uint4 ph, pl;
                    if (K == kSquare) {
                        ph = *reinterpret_cast<const uint4*>(own + at);
                        pl = *reinterpret_cast<const uint4*>(own + p.o_plane + at);
                    }
                    uint32_t w[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float v = acc[8 * k + q] * kHeldInv;
                        if (K == kSquare) {
                            const uint32_t h2 = q < 2 ? ph.x : q < 4 ? ph.y : q < 6 ? ph.z : ph.w;
                            const uint32_t l2 = q < 2 ? pl.x : q < 4 ? pl.y : q < 6 ? pl.z : pl.w;
                            v = p.c * v + p.b * joined(h2 >> (q & 1 ? 16 : 0), l2 >> (q & 1 ? 16 : 0));
                            if (C + q == R && R < p.m) v += p.a * kHeld;
                        }
                        w[q] = split(v);
                    }
                    uint4 hi, lo;
                    planes_of(w, hi, lo);
                    *reinterpret_cast<uint4*>(out + at) = hi;
                    *reinterpret_cast<uint4*>(out + p.o_plane + at) = lo;
                    if (kSym && (C >> 7) < i) {
                        // the block above the diagonal: rows and columns change places.  Two lanes exchange a value of two columns,
                        // so that each has two neighbours of one row
                        const bool odd = lane & 1;
#pragma unroll
                        for (int q = 0; q < 8; q += 2) {
                            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? w[q] : w[q + 1], 1);
                            const uint32_t x = odd ? other : w[q], y = odd ? w[q + 1] : other;
                            const int r = C + q + (odd ? 1 : 0), c = R & ~1;
                            const int64_t to = (int64_t(r >> 7) * p.o_panels + (c >> 6)) * kPanel + in_panel(r & 127, c & 63);
                            *reinterpret_cast<uint32_t*>(out + to) = __byte_perm(x, y, 0x5410);
                            *reinterpret_cast<uint32_t*>(out + p.o_plane + to) = __byte_perm(x, y, 0x7632);
                        }
                    }
                }
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == 9) {
        fence_after();
        tmem_free(tmem, L::cols);
    }
}

// ------------------------------------------------------------------------------------ on chip
//
// A cluster has a matrix, each of its blocks up to 256 of X's columns (4 panels) and all of P.  P's terms are summed over the
// cluster: the blocks' partial sums lie where P will be, each block adds up some rows and writes them to all.

constexpr int kChipThreads = 288, kChipPanels = 4;
constexpr int kChipSmem = 2 * kChipPanels * kPanel + 4 * kPanel + 1024;

struct Chip {
    Side g, out;
    int panels;  // of a block
    int steps;
    float a, b, c, scale;
    double eps;
    bool vec;
};

template <typename T>
__global__ void __launch_bounds__(kChipThreads, 1) chip_kernel(const Chip p, const T* gp, T* op) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t s_bar;
    __shared__ uint32_t s_tmem;
    __shared__ int s_dead;
    __shared__ double s_sum[9], s_norm;
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* xs = smem + 4 * kPanel;  // P: hi panels 0, 1, lo 0, 1; X: hi panels, lo panels
    const uint32_t sp = own_offset(uniform(smem_u32(smem))), sx = sp + 4 * kPanel;  // for descriptors
    const int warp = uniform(int(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = int(cluster.num_blocks()), rank = int(cluster.block_rank());
    const int matrix = blockIdx.x / blocks;
    const T* g = gp + int64_t(matrix) * p.g.matrix;
    T* out = op + int64_t(matrix) * p.out.matrix;
    const int c0 = rank * p.panels * 64, width = p.panels * 64;  // this block's columns
    const uint32_t x_plane = uint32_t(p.panels * kPanel), p_plane = 2 * kPanel;
    const uint32_t bar = smem_u32(&s_bar);
    if (threadIdx.x == 0) {
        s_dead = 0;
        bar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 8) tmem_alloc(smem_u32(&s_tmem), 512);

    // the norm, over the cluster
    Squares sq;
    const int cols = max(0, min(width, p.g.n - c0));
    for (int i = threadIdx.x; i < p.g.m * cols; i += kChipThreads) {
        const int u = p.g.turned ? i / p.g.m : i / cols, v = p.g.turned ? i - u * p.g.m : i - u * cols;
        sq.add(widen(g[p.g.at(p.g.turned ? v : u, c0 + (p.g.turned ? u : v))]));
    }
    const double w_sum = warp_sum(sq.total());
    if (lane == 0) s_sum[warp] = w_sum;
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = uniform(*reinterpret_cast<volatile uint32_t*>(&s_tmem));
    if (threadIdx.x == 0) {
        double t = 0;
        for (int w = 0; w < 9; ++w) t += s_sum[w];
        s_norm = t;
    }
    if (blocks > 1) cluster.sync();
    else __syncthreads();
    double total = 0;
    for (int b = 0; b < blocks; ++b) total += *cluster.map_shared_rank(&s_norm, b);
    const Factor inv(total, p.eps);

    // X_0's planes: 8 columns of a row at a time
    for (int i = threadIdx.x; i < 128 * p.panels * 8; i += kChipThreads) {
        const int r = p.g.turned ? i & 127 : i / (p.panels * 8), k = p.g.turned ? i >> 7 : i - r * (p.panels * 8);
        uint32_t w[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int c = c0 + k * 8 + q;
            w[q] = split(r < p.g.m && c < p.g.n ? inv.of(widen(g[p.g.at(r, c)])) * kHeld : 0.f);
        }
        uint4 hi, lo;
        planes_of(w, hi, lo);
        const uint32_t at = uint32_t(k >> 3) * kPanel + in_panel(r, (k & 7) * 8);
        *reinterpret_cast<uint4*>(xs + at) = hi;
        *reinterpret_cast<uint4*>(xs + x_plane + at) = lo;
    }
    volatile int* dead = &s_dead;
    unsigned* status = &ortho_status_word;
    const int quad = warp & 3, half = (warp >> 2) & 1, row = quad * 32 + lane;
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    const uint32_t lead = warp == 8 ? elect_lane() : 0;
    const int k16 = (p.g.m + 15) / 16;  // of a sum over the rows
    const uint32_t id_p = mma_desc<__half>(128, false), id_x = mma_desc<__half>(width, true);
    const int c16 = max(1, (cols + 15) / 16);  // of a sum over this block's columns; one at least: zeros
    uint32_t phase = 0;
    bool ok = true;
    // all writes of operands are done; the instructions that `issue` forms run, and everyone waits for them
    auto product = [&](auto issue) {
        fence_async_all();
        fence_before();
        ok = __syncthreads_and(ok);  // after a wait that was given up the block goes on to the end, for the others' sake
        if (!ok) return;
        if (warp == 8) {
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
    // columns c .. c + 31 of a product of n instructions
    auto sums = [&](int c, int n, bool wide, float (&v)[32]) {
        float u[32];
        const uint32_t at = uint32_t(c) + lanes;
        tmem_ld32(tmem + at, v);
        tmem_ld32(tmem + 256 + at, u);
        tmem_wait_ld(v);
        tmem_wait_ld(u);
        const float f0 = uncut(wide ? n : (n + 2) / 3);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = fmaf(v[i], f0, u[i] * kLoInv);
        if (!wide)
            for (int a = 1; a < min(n, 3); ++a) {
                tmem_ld32(hi_at(a) + at, u);
                tmem_wait_ld(u);
                const float f = uncut((n + 2 - a) / 3);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = fmaf(u[i], f, v[i]);
            }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= kHeldInv;
    };
    auto write = [&](unsigned char* to, uint32_t plane, int r, int c, const float* v) {
        uint32_t w[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = split(v[q]);
        uint4 hi, lo;
        planes_of(w, hi, lo);
        const uint32_t at = uint32_t(c >> 6) * kPanel + in_panel(r, c & 63);
        *reinterpret_cast<uint4*>(to + at) = hi;
        *reinterpret_cast<uint4*>(to + plane + at) = lo;
    };
    for (int step = 0; step < p.steps; ++step) {
        // P = X X^T
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
            if (warp < 8)
                for (int b = 0; b < 2; ++b) {
                    const int c = half * 64 + b * 32;
                    float v[32];
                    sums(c, c16, false, v);
#pragma unroll
                    for (int k = 0; k < 4; ++k) write(smem, p_plane, row, c + 8 * k, v + 8 * k);
                }
        } else {
            float* part = reinterpret_cast<float*>(smem);  // [128][128], 16-byte chunks of a row exchanged by its number
            auto at = [](int r, int chunk) { return r * 128 + ((chunk ^ (r & 31)) << 2); };
            if (warp < 8)
                for (int b = 0; b < 2; ++b) {
                    const int c = half * 64 + b * 32;
                    float v[32];
                    sums(c, c16, false, v);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<float4*>(part + at(row, c / 4 + k)) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
            cluster.sync();
            const int rows = 128 / blocks;
            float v[4][8];  // up to 4 chunks of 8 values a thread (2 blocks)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = threadIdx.x + u * 256;
                if (warp < 8 && i < rows * 16) {
                    const int r = rank * rows + (i >> 4), chunk = (i & 15) * 2;
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[u][q] = 0.f;
                    for (int b = 0; b < blocks; ++b) {
                        const float* other = cluster.map_shared_rank(part, b);
                        const float4 x = *reinterpret_cast<const float4*>(other + at(r, chunk)),
                                     y = *reinterpret_cast<const float4*>(other + at(r, chunk + 1));
                        v[u][0] += x.x, v[u][1] += x.y, v[u][2] += x.z, v[u][3] += x.w;
                        v[u][4] += y.x, v[u][5] += y.y, v[u][6] += y.z, v[u][7] += y.w;
                    }
                }
            }
            cluster.sync();
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = threadIdx.x + u * 256;
                if (warp < 8 && i < rows * 16)
                    for (int b = 0; b < blocks; ++b)
                        write(cluster.map_shared_rank(smem, b), p_plane, rank * rows + (i >> 4), (i & 15) * 8, v[u]);
            }
            fence_async_all();
            cluster.sync();
        }
        // M = a I + b P + c P P, where P was
        product([&] {
            for (int k = 0; k < k16; ++k) {
                const uint32_t x = sp + uint32_t(k >> 2) * kPanel;
                const uint64_t h = desc_cols(x, k & 3), l = desc_cols(x + p_plane, k & 3);
                mma_ss(lead, hi_at(k), h, h, id_p, k > 2);
                mma_ss(lead, tmem + 256, h, l, id_p, k > 0);
                mma_ss(lead, tmem + 256, l, h, id_p, true);
            }
        });
        if (warp < 8)
            for (int b = 0; b < 2; ++b) {
                const int c = half * 64 + b * 32;
                float v[32];
                sums(c, k16, false, v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t from = uint32_t(half) * kPanel + in_panel(row, b * 32 + 8 * k);
                    const uint4 ph = *reinterpret_cast<const uint4*>(smem + from), pl = *reinterpret_cast<const uint4*>(smem + p_plane + from);
                    const uint32_t h2[4] = {ph.x, ph.y, ph.z, ph.w}, l2[4] = {pl.x, pl.y, pl.z, pl.w};
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float& t = v[8 * k + q];
                        t = p.c * t + p.b * joined(h2[q >> 1] >> (q & 1 ? 16 : 0), l2[q >> 1] >> (q & 1 ? 16 : 0));
                        if (c + 8 * k + q == row && row < p.g.m) t += p.a * kHeld;
                    }
                    write(smem, p_plane, row, c + 8 * k, v + 8 * k);
                }
            }
        // X = M X
        product([&] {
            for (int k = 0; k < k16; ++k) {
                const uint32_t m = sp + uint32_t(k >> 2) * kPanel;
                const uint64_t mh = desc_cols(m, k & 3), ml = desc_cols(m + p_plane, k & 3);
                const uint64_t xh = desc_rows(sx, k), xl = desc_rows(sx + x_plane, k);
                mma_ss(lead, width > 128 ? tmem : hi_at(k), mh, xh, id_x, k > (width > 128 ? 0 : 2));
                mma_ss(lead, tmem + 256, mh, xl, id_x, k > 0);
                mma_ss(lead, tmem + 256, ml, xh, id_x, true);
            }
        });
        if (warp < 8)
            for (int b = half; b < p.panels * 2; b += 2) {
                float v[32];
                sums(32 * b, k16, width > 128, v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (step + 1 < p.steps) {
                        write(xs, x_plane, row, 32 * b + 8 * k, v + 8 * k);
                    } else {
                        float o[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) o[q] = v[8 * k + q] * (kHeldInv * p.scale);
                        give<T>(p.out, out, p.vec, row, c0 + 32 * b + 8 * k, o);
                    }
                }
            }
    }
    fence_before();
    __syncthreads();
    if (warp == 8) {
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
    z.fits = z.m <= 128 && z.n <= 64 * kChipPanels * 8;
    z.chip = z.fits && s.steps > 0;
    const int panels = up(z.n, 64) / 64;
    z.chip_blocks = 1;
    while (z.chip_blocks < 8 && panels > z.chip_blocks * kChipPanels) z.chip_blocks *= 2;
    z.chip_panels = (panels + z.chip_blocks - 1) / z.chip_blocks;
    return z;
}

struct Parts {
    double* norm;
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
    p.norm = reinterpret_cast<double*>(take(b * kNormBlocks * 8));
    if (!z.fits) {
        p.x[0] = take(b * 2 * z.x_plane);
        p.x[1] = take(b * 2 * z.x_plane);
        p.p = take(b * 2 * z.p_plane);
        p.q = take(b * 2 * z.p_plane);
    }
    p.bytes = used;
    return p;
}

template <typename... P, typename... Q>
cudaError_t launch(void (*k)(P...), int64_t blocks, int threads, int cluster, size_t smem, cudaStream_t st, Q... args) {
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(unsigned(blocks));
    c.blockDim = dim3(unsigned(threads));
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = unsigned(cluster);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k, static_cast<P>(args)...);
}

int sym_tiles(int blocks, int bn) {
    int t = 0;
    for (int i = 0; i < blocks; ++i) t += i / (bn / 128) + 1;
    return t;
}

// One product of every matrix (T: the type of kLast's result).  Tiles of 256 columns where they fill the card: they read a third less of the operands than those of
// 128, which give twice the blocks.
template <Kind K, typename T>
cudaError_t product(Product p, int matrices, int columns, int sms, cudaStream_t st) {
    constexpr bool kSym = K == kGram || K == kSquare;
    auto tiles = [&](int bn) { return kSym ? sym_tiles(p.blocks, bn) : p.blocks * (up(columns, bn) / bn); };
    const bool wide = int64_t(tiles(256)) * matrices >= sms * 3 / 4;
    p.tiles = tiles(wide ? 256 : 128);
    int splits = 1;  // of a long sum, where there are few tiles
    if (K == kGram)
        while (splits < 8 && int64_t(p.tiles) * matrices * splits * 2 <= sms && p.k_panels >= splits * 2 * 4) splits *= 2;
    const int64_t grid = int64_t(p.tiles) * matrices * splits;
    return wide ? launch(product_kernel<256, K, T>, grid, kThreads, splits, Tile<256>::smem, st, p)
                : launch(product_kernel<128, K, T>, grid, kThreads, splits, Tile<128>::smem, st, p);
}

template <typename T>
cudaError_t run(const OrthoShape& s, const void* gp, void* op, void* ws, int sms, cudaStream_t st) {
    const Sizes z = sizes_of(s);
    const Parts w = parts_of(s, z, ws);
    const T* g = static_cast<const T*>(gp);
    T* out = static_cast<T*>(op);
    const Side in = {z.m, z.n, z.turned, s.g_matrix, s.g_row}, to = {z.m, z.n, z.turned, s.o_matrix, s.o_row};
    const bool vec = ((reinterpret_cast<uintptr_t>(op) | uintptr_t(s.o_row) * sizeof(T) | uintptr_t(s.o_matrix) * sizeof(T)) & 15u) == 0;
    if (z.chip) {
        const Chip c = {in, to, z.chip_panels, s.steps, float(s.a), float(s.b), float(s.c), float(s.scale), s.eps, vec};
        return launch(chip_kernel<T>, int64_t(s.n_matrices) * z.chip_blocks, kChipThreads, z.chip_blocks, kChipSmem, st, c, g, out);
    }
    const int parts = std::min(kNormBlocks, s.rows);
    norm_kernel<T><<<dim3(parts, s.n_matrices), 512, 0, st>>>(s.rows, s.cols, s.g_matrix, s.g_row, g, w.norm);
    if (s.steps == 0) {
        scale_kernel<T><<<dim3(std::min(s.rows, 1024), s.n_matrices), 256, 0, st>>>(s.rows, s.cols, s.g_matrix, s.g_row, s.o_matrix, s.o_row,
                                                                                   float(s.scale), g, w.norm, parts, s.eps, out);
        return cudaGetLastError();
    }
    take_kernel<T><<<dim3(z.x_panels, z.blocks * 2, s.n_matrices), 256, 0, st>>>(in, g, w.norm, parts, s.eps, z.x_panels, z.x_plane, w.x[0]);
    cudaError_t e = cudaGetLastError();
    for (int i = 0; i < s.steps && e == cudaSuccess; ++i) {
        const char* x = w.x[i & 1];
        Product p = {};
        p.blocks = z.blocks, p.m = z.m;
        p.a = float(s.a), p.b = float(s.b), p.c = float(s.c);
        p.A = p.B = x, p.a_plane = p.b_plane = z.x_plane, p.a_panels = p.b_panels = z.x_panels;
        p.out = w.p, p.o_plane = z.p_plane, p.o_panels = z.p_panels;
        p.k_panels = up(z.n, 64) / 64;
        e = product<kGram, float>(p, s.n_matrices, z.m, sms, st);
        if (e != cudaSuccess) break;
        p.A = p.B = p.own = w.p, p.a_plane = p.b_plane = z.p_plane, p.a_panels = p.b_panels = z.p_panels;
        p.out = w.q;
        p.k_panels = up(z.m, 64) / 64;
        e = product<kSquare, float>(p, s.n_matrices, z.m, sms, st);
        if (e != cudaSuccess) break;
        p.A = w.q, p.B = x, p.b_plane = z.x_plane, p.b_panels = z.x_panels;
        p.out = w.x[(i + 1) & 1], p.o_plane = z.x_plane, p.o_panels = z.x_panels;
        p.side = to, p.scale = float(s.scale), p.vec = vec, p.result = out;
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
