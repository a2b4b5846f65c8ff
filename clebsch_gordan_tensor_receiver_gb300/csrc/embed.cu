// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//     out[t][c][i] = scale table[index[t]][c] for i = column, 0 for the other components
//     d_table[r][c] = scale sum over the tokens t with index[t] = r of d_out[t][c][column]
//
// Tokens whose index is not a row of the table (padding) give zeros and add to no row.
//
// Bound by memory.  The gradient sorts the tokens by row (stable, so that a row's tokens are added in their order), cuts the
// sorted tokens into pieces of equal length, however the rows lie, and sums each piece in fp32 registers.  A row whose tokens lie
// in one piece is written by it; the others are added up from the pieces' sums, in the pieces' order.
#include <algorithm>
#include <cstdint>

#include "elem.h"
#include "plan.h"

namespace uvu {
namespace {

constexpr int kThreads = 256;
constexpr int kDigit = 8, kBins = 1 << kDigit;  // of the sort's passes
constexpr int kKeys = 8;                        // keys of a thread and tile
constexpr int kTile = kThreads * kKeys;
constexpr int kMaxBlocks = 512;                 // of a pass
constexpr int kPiece = 32;                      // tokens of a piece

// A row that is not the table's is one past its last, which sorts it behind all others.
__device__ __forceinline__ uint32_t row_of(int32_t i, uint32_t rows) { return uint32_t(i) < rows ? uint32_t(i) : rows; }

template <typename T>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(int64_t tokens, uint32_t rows, int channels, int inner, int column,
                                                             float scale, const int32_t* index, const T* table, T* out) {
    const int width = channels * inner;
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        const uint32_t r = row_of(index[t], rows);
        for (int e = threadIdx.x; e < width; e += kThreads) {
            const int c = e / inner;
            const float v = r < rows && e - c * inner == column ? widen(table[int64_t(r) * channels + c]) * scale : 0.f;
            out[t * width + e] = narrow<T>(v);
        }
    }
}

// ------------------------------------------------------------------------------------- the sort
//
// Stable passes over 8 bits of the row, lowest first.  A block has `tiles` consecutive tiles of the keys; counts [bin][block].

__global__ void __launch_bounds__(kThreads) count_kernel(int64_t n, uint32_t rows, const int32_t* index, const uint32_t* keys, int shift,
                                                         int tiles, uint32_t* counts) {
    __shared__ uint32_t s[kBins];
    s[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * tiles * kTile, end = min(first + int64_t(tiles) * kTile, n);
    for (int64_t i = first + threadIdx.x; i < end; i += kThreads) {
        const uint32_t key = keys ? keys[i] : row_of(index[i], rows);
        atomicAdd(s + ((key >> shift) & (kBins - 1)), 1u);
    }
    __syncthreads();
    counts[int64_t(threadIdx.x) * gridDim.x + blockIdx.x] = s[threadIdx.x];
}

// Exclusive sums of a bin's counts over the blocks, and the bin's total: one block per bin.
__global__ void __launch_bounds__(kMaxBlocks) bins_kernel(int blocks, uint32_t* counts, uint32_t* totals) {
    __shared__ uint32_t s[kMaxBlocks];
    const int i = threadIdx.x;
    uint32_t* row = counts + int64_t(blockIdx.x) * blocks;
    const uint32_t own = i < blocks ? row[i] : 0;
    s[i] = own;
    for (int d = 1; d < kMaxBlocks; d *= 2) {
        __syncthreads();
        const uint32_t v = i >= d ? s[i - d] : 0;
        __syncthreads();
        s[i] += v;
    }
    if (i < blocks) row[i] = s[i] - own;
    if (i == kMaxBlocks - 1) totals[blockIdx.x] = s[i];
}

__global__ void __launch_bounds__(kThreads) place_kernel(int64_t n, uint32_t rows, const int32_t* index, const uint32_t* keys,
                                                         const int32_t* ids, int shift, int tiles, const uint32_t* counts,
                                                         const uint32_t* totals, uint32_t* keys_out, int32_t* ids_out) {
    __shared__ uint32_t s_base[kBins], s_scan[kBins], s_warp[kThreads / 32][kBins];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    s_scan[tid] = totals[tid];
    for (int d = 1; d < kBins; d *= 2) {
        __syncthreads();
        const uint32_t v = tid >= d ? s_scan[tid - d] : 0;
        __syncthreads();
        s_scan[tid] += v;
    }
    __syncthreads();
    s_base[tid] = s_scan[tid] - totals[tid] + counts[int64_t(tid) * gridDim.x + blockIdx.x];
    for (int tile = 0; tile < tiles; ++tile) {
        const int64_t first = (int64_t(blockIdx.x) * tiles + tile) * kTile;
        if (first >= n) break;
        for (int w = 0; w < kThreads / 32; ++w) s_warp[w][tid] = 0;
        __syncthreads();
        uint32_t key[kKeys], rank[kKeys];
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {  // a warp's keys lie together, 32 at a time
            const int64_t i = first + warp * (kKeys * 32) + k * 32 + lane;
            const bool live = i < n;
            key[k] = live ? (keys ? keys[i] : row_of(index[i], rows)) : 0;
            const uint32_t bin = live ? (key[k] >> shift) & (kBins - 1) : kBins;
            const uint32_t same = __match_any_sync(0xffffffffu, bin);
            const uint32_t before = live ? s_warp[warp][bin] : 0;
            rank[k] = before + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (live && lane == 31 - __clz(same)) s_warp[warp][bin] = rank[k] + 1;
            __syncwarp();
        }
        __syncthreads();
        uint32_t run = s_base[tid];  // of bin tid: where each warp's keys begin
        for (int w = 0; w < kThreads / 32; ++w) {
            const uint32_t c = s_warp[w][tid];
            s_warp[w][tid] = run;
            run += c;
        }
        s_base[tid] = run;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kKeys; ++k) {
            const int64_t i = first + warp * (kKeys * 32) + k * 32 + lane;
            if (i < n) {
                const uint32_t to = s_warp[warp][(key[k] >> shift) & (kBins - 1)] + rank[k];
                keys_out[to] = key[k];
                ids_out[to] = ids ? ids[i] : int32_t(i);
            }
        }
        __syncthreads();
    }
}

// starts[r]: the first sorted token whose row is r or more, for r = 0 .. rows.
__global__ void starts_kernel(int64_t n, uint32_t rows, const uint32_t* keys, int32_t* starts) {
    for (int64_t r = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; r <= rows; r += int64_t(gridDim.x) * blockDim.x) {
        int64_t lo = 0, hi = n;
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (keys[mid] < uint32_t(r)) lo = mid + 1;
            else hi = mid;
        }
        starts[r] = int32_t(lo);
    }
}

// ------------------------------------------------------------------------------------- the sums

// A block has a piece of the sorted tokens.  part [piece][2][channels]: the sum of the row that the piece begins with, where that
// row also lies in the piece before or after, and of the one that it ends with, where it goes on behind.
template <typename T>
__global__ void __launch_bounds__(kThreads) piece_kernel(int64_t n, uint32_t rows, int channels, int inner, int column, float scale,
                                                         const uint32_t* keys, const int32_t* ids, const int32_t* starts, const T* dout,
                                                         T* dtable, float* part) {
    const int64_t p0 = int64_t(blockIdx.x) * kPiece, p1 = min(min(p0 + kPiece, n), int64_t(starts[rows]));
    if (p0 >= p1) return;
    const int64_t width = int64_t(channels) * inner;
    for (int c = threadIdx.x; c < channels; c += kThreads) {
        float sum = 0.f;
        for (int64_t p = p0; p < p1; ++p) {
            const uint32_t r = keys[p];
            sum += widen(dout[int64_t(ids[p]) * width + int64_t(c) * inner + column]);
            if (p + 1 == p1 || keys[p + 1] != r) {
                const bool head = starts[r] < p0, tail = starts[r + 1] > p1;
                if (!head && !tail)
                    dtable[int64_t(r) * channels + c] = narrow<T>(sum * scale);
                else
                    part[(int64_t(blockIdx.x) * 2 + (head ? 0 : 1)) * channels + c] = sum;
                sum = 0.f;
            }
        }
    }
}

// The rows without tokens, and those of several pieces.
template <typename T>
__global__ void __launch_bounds__(kThreads) join_kernel(uint32_t rows, int channels, float scale, const int32_t* starts, const float* part,
                                                        T* dtable) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int64_t a = starts[r], b = starts[r + 1];
        const int64_t first = a / kPiece, last = (b - 1) / kPiece;
        if (a < b && first == last) continue;
        for (int c = threadIdx.x; c < channels; c += kThreads) {
            float sum = 0.f;
            if (a < b) {
                sum = part[(first * 2 + 1) * channels + c];
                float lost = 0.f;  // what the additions so far cut off: a frequent row has thousands of pieces
                for (int64_t p = first + 1; p <= last; ++p) {
                    const float v = part[p * 2 * channels + c], t = sum + v, back = t - sum;
                    lost += (sum - (t - back)) + (v - back);
                    sum = t;
                }
                sum += lost;
            }
            dtable[r * channels + c] = narrow<T>(sum * scale);
        }
    }
}

struct SortPlan {
    int passes, tiles, blocks;
};
SortPlan sort_plan(const EmbedShape& s) {
    SortPlan p;
    p.passes = 1;
    while (p.passes < 4 && (int64_t(s.rows) >> (p.passes * kDigit)) > 0) ++p.passes;
    const int64_t tiles = (s.tokens + kTile - 1) / kTile;
    p.tiles = int((tiles + kMaxBlocks - 1) / kMaxBlocks);
    p.blocks = int((tiles + p.tiles - 1) / p.tiles);
    return p;
}

struct Work {
    uint32_t *keys[2], *counts, *totals;
    int32_t *ids[2], *starts;
    float* part;
    size_t bytes;
};
Work work_of(const EmbedShape& s, void* ws) {
    const SortPlan p = sort_plan(s);
    char* at = static_cast<char*>(ws);
    size_t used = 0;
    auto take = [&](size_t b) {
        char* r = at + used;
        used += align256(b);
        return r;
    };
    Work w;
    for (int i = 0; i < 2; ++i) {
        w.keys[i] = reinterpret_cast<uint32_t*>(take(size_t(s.tokens) * 4));
        w.ids[i] = reinterpret_cast<int32_t*>(take(size_t(s.tokens) * 4));
    }
    w.counts = reinterpret_cast<uint32_t*>(take(size_t(p.blocks) * kBins * 4));
    w.totals = reinterpret_cast<uint32_t*>(take(kBins * 4));
    w.starts = reinterpret_cast<int32_t*>(take((size_t(s.rows) + 1) * 4));
    w.part = reinterpret_cast<float*>(take(size_t((s.tokens + kPiece - 1) / kPiece) * 2 * s.channels * 4));
    w.bytes = used;
    return w;
}

template <typename T>
cudaError_t bwd(const EmbedShape& s, const int32_t* index, const void* dout, void* dtable, void* ws, int sms, cudaStream_t st) {
    const SortPlan p = sort_plan(s);
    const Work w = work_of(s, ws);
    const uint32_t rows = uint32_t(s.rows);
    const uint32_t* keys = nullptr;
    const int32_t* ids = nullptr;
    for (int i = 0; i < p.passes; ++i) {
        count_kernel<<<p.blocks, kThreads, 0, st>>>(s.tokens, rows, index, keys, i * kDigit, p.tiles, w.counts);
        bins_kernel<<<kBins, kMaxBlocks, 0, st>>>(p.blocks, w.counts, w.totals);
        place_kernel<<<p.blocks, kThreads, 0, st>>>(s.tokens, rows, index, keys, ids, i * kDigit, p.tiles, w.counts, w.totals, w.keys[i & 1],
                                                    w.ids[i & 1]);
        keys = w.keys[i & 1];
        ids = w.ids[i & 1];
    }
    starts_kernel<<<unsigned(std::min<int64_t>((s.rows + 256) / 256, sms * 8)), 256, 0, st>>>(s.tokens, rows, keys, w.starts);
    piece_kernel<T><<<unsigned((s.tokens + kPiece - 1) / kPiece), kThreads, 0, st>>>(
        s.tokens, rows, s.channels, s.inner, s.column, float(s.scale), keys, ids, w.starts, static_cast<const T*>(dout),
        static_cast<T*>(dtable), w.part);
    join_kernel<T><<<unsigned(std::min<int64_t>(s.rows, sms * 16)), kThreads, 0, st>>>(rows, s.channels, float(s.scale), w.starts, w.part,
                                                                                      static_cast<T*>(dtable));
    return cudaGetLastError();
}

template <typename T>
cudaError_t fwd(const EmbedShape& s, const int32_t* index, const void* table, void* out, int sms, cudaStream_t st) {
    embed_fwd_kernel<T><<<unsigned(std::min<int64_t>(s.tokens, sms * 16)), kThreads, 0, st>>>(
        s.tokens, uint32_t(s.rows), s.channels, s.inner, s.column, float(s.scale), index, static_cast<const T*>(table),
        static_cast<T*>(out));
    return cudaGetLastError();
}

}  // namespace

size_t embed_workspace(const EmbedShape& s) { return s.tokens == 0 || s.rows == 0 ? 0 : work_of(s, nullptr).bytes; }

cudaError_t launch_embed_fwd(const EmbedShape& s, const int32_t* index, const void* table, void* out, int sms, cudaStream_t st) {
    switch (s.dtype) {
        case UVU_F32: return fwd<float>(s, index, table, out, sms, st);
        case UVU_BF16: return fwd<__nv_bfloat16>(s, index, table, out, sms, st);
        case UVU_F16: return fwd<__half>(s, index, table, out, sms, st);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_embed_bwd(const EmbedShape& s, const int32_t* index, const void* dout, void* dtable, void* ws, int sms,
                             cudaStream_t st) {
    if (s.tokens == 0) return cudaMemsetAsync(dtable, 0, size_t(s.rows) * s.channels * (s.dtype == UVU_F32 ? 4 : 2), st);
    switch (s.dtype) {
        case UVU_F32: return bwd<float>(s, index, dout, dtable, ws, sms, st);
        case UVU_BF16: return bwd<__nv_bfloat16>(s, index, dout, dtable, ws, sms, st);
        case UVU_F16: return bwd<__half>(s, index, dout, dtable, ws, sms, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace uvu
