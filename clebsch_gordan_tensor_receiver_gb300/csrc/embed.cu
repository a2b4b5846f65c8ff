// Embedding lookup with scaling, and its gradient by sorted tokens.
//
//     out[t][c][i] = scale table[index[t]][c] for i = column, 0 for the other components
//     d_table[r][c] = scale sum over the tokens t with index[t] = r of d_out[t][c][column]
//
// Tokens whose index is not a row of the table (padding) give zeros and add to no row.
//
// Bound by memory: the lookup writes out once (the table's used rows come from the L2 cache), in 16-byte vectors (300,007 x 512 in f16: 52 us,
// 5.9 TB/s).
//
// The gradient adds no two threads' sums by atomic instructions, whose order would change the result.  It sorts the tokens by row (stable,
// so that a row's tokens are added in their order), cuts the sorted tokens into pieces of equal length, however the rows lie,
// and sums each piece in fp32 registers, 8 rows of d_out on their way at a time.  A row whose tokens lie in one piece is
// written by it; one that goes on behind its piece is noted, and added up from the pieces' sums, in their order where it reaches up to 16
// more, else by 4 or 16 ways that take turns.  Rows without a token
// are zeros: the table is zeroed by blocks of the first kernel that the sort leaves idle.  300,007 x 512 of f16 into 119 rows: 88 us, 21 of
// them the sort; 16,384 tokens of a 65,536 x 1024 table in bf16: 61 us, 34 of them the sort in one block, beside which the table is zeroed.
#include <algorithm>
#include <cstdint>

#include "elem.h"
#include "plan.h"

namespace uvu {
namespace {

__device__ __forceinline__ void next_may_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ----------------------------------------------------------------------------------- the lookup

constexpr int kLookupTokens = 4;  // of a thread at a time: their table rows are on their way together

// Threads (x: vectors of an output row, y: tokens).  PLAIN: inner == 1, and a vector of out is one of the table.
template <typename T, int V, bool PLAIN>
__global__ void __launch_bounds__(256) embed_fwd_kernel(int64_t tokens, uint32_t rows, int channels, int inner, int column, float scale,
                                                        const int32_t* index, const T* table, T* out) {
    const int width = channels * inner, vecs = width / V;
    const int64_t t0 = int64_t(blockIdx.x) * blockDim.y * kLookupTokens + threadIdx.y;
    int32_t at[kLookupTokens];
#pragma unroll
    for (int k = 0; k < kLookupTokens; ++k) {
        const int64_t t = t0 + k * blockDim.y;
        at[k] = t < tokens ? index[t] : -1;
    }
    for (int c = blockIdx.y * blockDim.x + threadIdx.x; c < vecs; c += gridDim.y * blockDim.x) {
        // of this vector's values those that are `column` of their channel, and the first one's channel
        uint32_t hits = 0;
        int first = c * V;
        if (!PLAIN) {
            const int e = c * V, ch = e / inner, r = e - ch * inner;
            int h = column - r;
            first = ch;
            if (h < 0) h += inner, ++first;
            for (; h < V; h += inner) hits |= 1u << h;
        }
        Pack<T, V> o[kLookupTokens];
#pragma unroll
        for (int k = 0; k < kLookupTokens; ++k) {
            o[k].clear();
            if (uint32_t(at[k]) < rows) {
                const T* p = table + int64_t(at[k]) * channels + first;
                if (PLAIN) {
                    o[k] = *reinterpret_cast<const Pack<T, V>*>(p);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (hits >> i & 1) o[k].put(i, *p++);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kLookupTokens; ++k) {
            const int64_t t = t0 + k * blockDim.y;
            float v[V];
            o[k].get(v);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= scale;
            o[k].set(v);
            // what is not looked up is zero, and not minus zero under a negative scale
            if (uint32_t(at[k]) >= rows) o[k].clear();
            if (!PLAIN)
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (!(hits >> i & 1)) o[k].put(i, T(0.f));
            if (t < tokens) *reinterpret_cast<Pack<T, V>*>(out + t * width + int64_t(c) * V) = o[k];
        }
    }
}

// -------------------------------------------------------------------------------------- the sort
//
// Stable passes over 8 bits of the row, lowest first.  The first pass leaves padding out; behind it come `*valid` tokens.  Up to kOneBlock
// tokens, as many as its shared memory holds, one block makes all passes, else each pass is three kernels: the blocks' counts of each bin,
// their running sums, and the placing.  The whole gradient of 128 fp32 channels in one block and in three kernels a pass: 10,000 rows (two
// passes), 1024 tokens 16 and 20 us, 4096 tokens 21 and 26, 8192 tokens 28 and 33, 16,384 tokens 43 and 37; 119 rows (one), 4096 tokens 17
// and 17, 16,384 tokens 33 and 23.

constexpr int kThreads = 256;
constexpr int kDigit = 8, kBins = 1 << kDigit;
constexpr int kKeys = 8;                   // of a thread and tile
constexpr int kTile = kThreads * kKeys;
constexpr int kMaxBlocks = 512;            // of a pass; a block takes consecutive tiles
constexpr int kOneThreads = 1024, kOneKeys = 16, kOneBlock = kOneThreads * kOneKeys;
// Behind the two numbers of valid tokens those of the rows that go on behind the piece they begin in, by how far: see join_kernel.
constexpr int kChains = 2, kReaches = 3;
__device__ __forceinline__ constexpr int reach(int i) { return i == 0 ? 16 : 256; }  // pieces, of the first two
constexpr int kOneSmem = 2 * kOneBlock * 4 + 2 * kOneBlock * 2 + (kOneThreads / 32) * kBins * 4;

// Zeros over [p, p + bytes), by the blocks from `first` on of the grid.
__device__ __forceinline__ void zero(unsigned char* p, int64_t bytes, int first) {
    const int64_t threads = int64_t(gridDim.x - first) * blockDim.x, me = int64_t(blockIdx.x - first) * blockDim.x + threadIdx.x;
    const int64_t head = min(bytes, int64_t((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15)), vecs = (bytes - head) / 16;
    for (int64_t i = me; i < head; i += threads) p[i] = 0;
    uint4* v = reinterpret_cast<uint4*>(p + head);
    for (int64_t i = me; i < vecs; i += threads) v[i] = make_uint4(0, 0, 0, 0);
    for (int64_t i = head + vecs * 16 + me; i < bytes; i += threads) p[i] = 0;
}

// Ranks of a warp's next 32 keys within their bins, after those that `seen` (of the warp) counts; live: the lane has a key.  The lanes of a
// bin find one another bit by bit.
__device__ __forceinline__ uint32_t warp_rank(uint32_t* seen, uint32_t bin, bool live, int lane) {
    uint32_t same = __ballot_sync(0xffffffffu, live);
#pragma unroll
    for (int b = 0; b < kDigit; ++b) {
        const bool set = bin >> b & 1;
        const uint32_t with = __ballot_sync(0xffffffffu, set);
        same &= set ? with : ~with;
    }
    const uint32_t rank = (live ? seen[bin] : 0) + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (live && lane == 31 - __clz(same)) seen[bin] = rank + 1;
    __syncwarp();
    return rank;
}
// Sum of the values of the threads before this one, over the block's first kBins threads (all threads call it).
__device__ __forceinline__ uint32_t before(uint32_t v, uint32_t* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t run = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += u;
    }
    if (lane == 31 && warp < kBins / 32) s_warp[warp] = run;
    __syncthreads();
    for (int w = 0; w < kBins / 32; ++w)
        if (w < warp) run += s_warp[w];
    return run - v;
}

// A large table is zeroed beside the sort, not by blocks of it, which fill an SM each with their shared memory: it begins when the sort
// has begun, and ends after it.
constexpr int64_t kLargeTable = 4 << 20;
__global__ void __launch_bounds__(kThreads) zero_kernel(unsigned char* table, int64_t bytes) {
    next_may_begin();
    zero(table, bytes, 0);
    wait_for_last();
}

__global__ void __launch_bounds__(kOneThreads) sort_kernel(int n, uint32_t rows, int passes, const int32_t* index, uint32_t* keys_out,
                                                           int32_t* ids_out, int32_t* valid, unsigned char* table, int64_t table_bytes) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ uint32_t s_sum[kBins / 32];
    __shared__ int s_valid;
    next_may_begin();
    if (blockIdx.x > 0) return zero(table, table_bytes, 1);
    uint32_t* s_key = reinterpret_cast<uint32_t*>(smem);                              // [2][kOneBlock]
    uint16_t* s_id = reinterpret_cast<uint16_t*>(s_key + 2 * kOneBlock);              // [2][kOneBlock]
    uint32_t* s_seen = reinterpret_cast<uint32_t*>(s_id + 2 * kOneBlock);             // [warps][kBins]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int m = n;
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * kDigit, from = (pass & 1) * kOneBlock, to = kOneBlock - from;
        for (int i = tid; i < kOneThreads / 32 * kBins; i += kOneThreads) s_seen[i] = 0;
        __syncthreads();
        uint32_t key[kOneKeys], rank[kOneKeys];
        const int rounds = (m + kOneThreads - 1) / kOneThreads, used = (m + rounds * 32 - 1) / max(1, rounds * 32);  // warps with keys
        auto place_of = [&](int k) { return k < rounds ? warp * (rounds * 32) + k * 32 + lane : m; };  // a warp's keys lie together
#pragma unroll
        for (int k = 0; k < kOneKeys; ++k) {
            const int i = place_of(k);
            key[k] = i >= m ? rows : pass == 0 ? uint32_t(index[i]) : s_key[from + i];
        }
#pragma unroll
        for (int k = 0; k < kOneKeys; ++k)
            if (k < rounds && warp < used) rank[k] = warp_rank(s_seen + warp * kBins, key[k] >> shift & (kBins - 1), key[k] < rows, lane);
        __syncthreads();
        // where each warp's keys of a bin begin
        uint32_t total = 0;
        if (tid < kBins)
            for (int w = 0; w < used; ++w) total += s_seen[w * kBins + tid];
        uint32_t run = before(total, s_sum);
        if (tid < kBins) {
            if (tid == kBins - 1) s_valid = int(run + total);
            for (int w = 0; w < used; ++w) {
                const uint32_t c = s_seen[w * kBins + tid];
                s_seen[w * kBins + tid] = run;
                run += c;
            }
        }
        __syncthreads();
        const bool last = pass == passes - 1;
#pragma unroll
        for (int k = 0; k < kOneKeys; ++k) {
            const int i = place_of(k);
            if (key[k] < rows) {
                const uint32_t p = s_seen[warp * kBins + (key[k] >> shift & (kBins - 1))] + rank[k];
                const int id = pass == 0 ? i : s_id[from + i];
                if (last) {
                    keys_out[p] = key[k];
                    ids_out[p] = id;
                } else {
                    s_key[to + p] = key[k];
                    s_id[to + p] = uint16_t(id);
                }
            }
        }
        m = s_valid;
        __syncthreads();
    }
    if (tid == 0) {
        valid[0] = m;
        for (int i = 0; i < kReaches; ++i) valid[kChains + i] = 0;
    }
}

// The keys of a pass: the indices, or what the last pass left.
struct Keys {
    int64_t n;
    uint32_t rows;
    const int32_t* index;   // first pass
    const uint32_t* keys;   // later ones, with their number
    const int32_t *ids, *valid;
    int shift, tiles;
    __device__ __forceinline__ int64_t count() const { return keys ? *valid : n; }
    __device__ __forceinline__ uint32_t key(int64_t i) const { return keys ? keys[i] : uint32_t(index[i]); }
    __device__ __forceinline__ uint32_t bin(uint32_t key) const { return key >> shift & (kBins - 1); }
};

// counts [bin][block].  Blocks from `blocks` on zero the table.
__global__ void __launch_bounds__(kThreads) count_kernel(const Keys k, int blocks, uint32_t* counts, unsigned char* table, int64_t table_bytes) {
    __shared__ uint32_t s[kBins];
    next_may_begin();
    if (int(blockIdx.x) >= blocks) return zero(table, table_bytes, blocks);
    s[threadIdx.x] = 0;
    __syncthreads();
    wait_for_last();
    const int64_t n = k.count(), first = int64_t(blockIdx.x) * k.tiles * kTile, end = min(first + int64_t(k.tiles) * kTile, n);
    for (int64_t i = first + threadIdx.x; i < end; i += kThreads) {
        const uint32_t key = k.key(i);
        if (key < k.rows) atomicAdd(s + k.bin(key), 1u);
    }
    __syncthreads();
    counts[int64_t(threadIdx.x) * blocks + blockIdx.x] = s[threadIdx.x];
}

// Running sums of a bin's counts over the blocks, and the bin's total: one block per bin.
__global__ void __launch_bounds__(kMaxBlocks) bins_kernel(int blocks, uint32_t* counts, uint32_t* totals) {
    __shared__ uint32_t s[kMaxBlocks / 32];
    next_may_begin();
    wait_for_last();
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    uint32_t* row = counts + int64_t(blockIdx.x) * blocks;
    const uint32_t own = i < blocks ? row[i] : 0;
    uint32_t run = own;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += u;
    }
    if (lane == 31) s[warp] = run;
    __syncthreads();
    for (int w = 0; w < kMaxBlocks / 32; ++w)
        if (w < warp) run += s[w];
    if (i < blocks) row[i] = run - own;
    if (i == kMaxBlocks - 1) totals[blockIdx.x] = run;
}

__global__ void __launch_bounds__(kThreads) place_kernel(const Keys k, const uint32_t* counts, const uint32_t* totals, uint32_t* keys_out,
                                                         int32_t* ids_out, int32_t* valid, int parity) {
    __shared__ uint32_t s_base[kBins], s_sum[kBins / 32], s_warp[kThreads / 32][kBins];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    next_may_begin();
    wait_for_last();
    const int64_t n = k.count();
    const uint32_t total = totals[tid], first_of = before(total, s_sum);
    if (blockIdx.x == 0 && tid == kBins - 1) {
        valid[parity] = int32_t(first_of + total);
        for (int i = 0; i < kReaches; ++i) valid[kChains + i] = 0;
    }
    s_base[tid] = first_of + counts[int64_t(tid) * gridDim.x + blockIdx.x];
    for (int tile = 0; tile < k.tiles; ++tile) {
        const int64_t first = (int64_t(blockIdx.x) * k.tiles + tile) * kTile;
        if (first >= n) break;
        for (int w = 0; w < kThreads / 32; ++w) s_warp[w][tid] = 0;
        uint32_t key[kKeys], rank[kKeys];
        bool live[kKeys];
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {  // a warp's keys lie together, 32 at a time
            const int64_t i = first + warp * (kKeys * 32) + j * 32 + lane;
            key[j] = i < n ? k.key(i) : 0;
            live[j] = i < n && key[j] < k.rows;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kKeys; ++j) rank[j] = warp_rank(s_warp[warp], k.bin(key[j]), live[j], lane);
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
        for (int j = 0; j < kKeys; ++j) {
            const int64_t i = first + warp * (kKeys * 32) + j * 32 + lane;
            if (live[j]) {
                const uint32_t to = s_warp[warp][k.bin(key[j])] + rank[j];
                keys_out[to] = key[j];
                ids_out[to] = k.ids ? k.ids[i] : int32_t(i);
            }
        }
        __syncthreads();
    }
}

// -------------------------------------------------------------------------------------- the sums

constexpr int kSumThreads = 128;
constexpr int kBatch = 8;  // rows of d_out on their way

struct Sums {
    int64_t pieces;
    int piece;            // tokens of one
    int channels, inner, column;
    float scale;
    const uint32_t* keys;
    const int32_t *ids, *valid;
    float* part;          // [piece][2][channels]
    int32_t *chains, *chain;  // the numbers of rows that go on behind the piece they begin in, and [3][pieces] these pieces, in any order
};

// Threads (x: vectors of channels, y: pieces).  part: the sum of the row that the piece begins with, where that row begins before it
// (whether or not it also ends behind it), and of one that begins in it and goes on behind.  V > 1: inner == 1.
template <typename T, int V>
__global__ void __launch_bounds__(kSumThreads) piece_kernel(const Sums s, const T* dout, T* dtable) {
    next_may_begin();
    wait_for_last();
    const int64_t piece = int64_t(blockIdx.x) * blockDim.y + threadIdx.y, n = *s.valid;
    const int64_t p0 = piece * s.piece, p1 = min(p0 + s.piece, n);
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * V;
    if (p0 >= p1 || c >= s.channels) return;
    const int64_t width = int64_t(s.channels) * s.inner;
    const T* from = dout + int64_t(c) * s.inner + s.column;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.f;
    uint32_t row = s.keys[p0];
    bool head = p0 > 0 && s.keys[p0 - 1] == row;
    auto flush = [&](bool on) {  // the row is summed, or goes on behind the piece
        if (head || on) {
            float* p = s.part + (piece * 2 + (head ? 0 : 1)) * s.channels + c;
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = sum[i];
        } else {
            float f[V];
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = sum[i] * s.scale;
            Pack<T, V> o;
            o.set(f);
            *reinterpret_cast<Pack<T, V>*>(dtable + int64_t(row) * s.channels + c) = o;
        }
    };
    for (int64_t p = p0; p < p1; p += kBatch) {
        uint32_t key[kBatch];
        Pack<T, V> v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (p + b < p1) {
                key[b] = s.keys[p + b];
                v[b] = *reinterpret_cast<const Pack<T, V>*>(from + int64_t(s.ids[p + b]) * width);
            }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (p + b < p1) {
                if (key[b] != row) {
                    flush(false);
                    row = key[b];
                    head = false;
#pragma unroll
                    for (int i = 0; i < V; ++i) sum[i] = 0.f;
                }
                float f[V];
                v[b].get(f);
#pragma unroll
                for (int i = 0; i < V; ++i) sum[i] += f[i];
            }
    }
    const bool on = p1 < n && s.keys[p1] == row;
    flush(on);
    if (on && !head && c == 0) {
        auto reaches = [&](int far) { return (piece + far) * s.piece < n && s.keys[(piece + far) * s.piece] == row; };
        const int which = !reaches(reach(0) + 1) ? 0 : !reaches(reach(1) + 1) ? 1 : 2;
        s.chain[which * s.pieces + atomicAdd(s.chains + which, 1)] = int32_t(piece);
    }
}

// The rows that go on behind the piece in which they begin.  A task is one of them and so many channels: 256 where it reaches a few
// pieces, else fewer, with the block's threads along the pieces too.
constexpr int kJoinThreads = 256;
template <int CHANNELS, typename T>
__device__ void join(const Sums& s, int64_t n, int64_t first, int c0, float* s_sum, T* dtable) {
    constexpr int kWays = kJoinThreads / CHANNELS;
    const int tid = threadIdx.x, way = tid / CHANNELS, lane = tid % CHANNELS, c = c0 + lane;
    const uint32_t row = s.keys[(first + 1) * s.piece];
    // the last piece that begins with the row: as many places at once as there are threads
    int64_t last = first + 1, span = (n + s.piece - 1) / s.piece - last;  // pieces last .. last + span - 1 may, the first does
    if (CHANNELS == kJoinThreads) span = min(span, int64_t(reach(0)));
    else if (CHANNELS == 64) span = min(span, int64_t(reach(1)));
    while (span > 1) {
        const int64_t step = (span + kJoinThreads - 1) / kJoinThreads;
        const bool same = tid * step < span && s.keys[(last + tid * step) * s.piece] == row;
        const int64_t skip = int64_t(__syncthreads_count(same) - 1) * step;  // sorted: those that begin with it come first
        last += skip;
        span = min(step, span - skip);
    }
    float sum = 0.f, lost = 0.f;  // what the additions cut off: a frequent row has thousands of pieces
    if (c < s.channels) {
        if (way == 0) sum = s.part[(first * 2 + 1) * s.channels + c];
#pragma unroll 8
        for (int64_t q = first + 1 + way; q <= last; q += kWays) {
            const float v = s.part[q * 2 * s.channels + c], t = sum + v, back = t - sum;
            lost += (sum - (t - back)) + (v - back);
            sum = t;
        }
    }
    if (fabsf(sum) <= 3.4028235e38f) sum += lost;  // an infinity stays one: what it cut off is NaN
    if (kWays > 1) {
        __syncthreads();  // the last task's sums have been read
        s_sum[way * CHANNELS + lane] = sum;
        __syncthreads();
        if (way == 0)
#pragma unroll
            for (int w = 1; w < kWays; ++w) sum += s_sum[w * CHANNELS + lane];
    }
    if (way == 0 && c < s.channels) dtable[int64_t(row) * s.channels + c] = narrow<T>(sum * s.scale);
}
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Sums s, T* dtable) {
    __shared__ float s_sum[kJoinThreads];
    wait_for_last();
    const int64_t n = *s.valid;
    const auto slabs = [&](int channels) { return (s.channels + channels - 1) / channels; };
    const int64_t far = int64_t(s.chains[2]) * slabs(16), middle = far + int64_t(s.chains[1]) * slabs(64),
                  all = middle + int64_t(s.chains[0]) * slabs(kJoinThreads);
    for (int64_t task = blockIdx.x; task < all; task += gridDim.x) {  // the longest first
        const int which = task < far ? 2 : task < middle ? 1 : 0, channels = which == 2 ? 16 : which == 1 ? 64 : kJoinThreads;
        const int64_t t = task - (which == 2 ? 0 : which == 1 ? far : middle), chain = t / slabs(channels);
        const int64_t first = s.chain[which * s.pieces + chain];
        const int c0 = int(t - chain * slabs(channels)) * channels;
        if (which == 2) join<16>(s, n, first, c0, s_sum, dtable);
        else if (which == 1) join<64>(s, n, first, c0, s_sum, dtable);
        else join<kJoinThreads>(s, n, first, c0, s_sum, dtable);
    }
}

// ----------------------------------------------------------------------------------------- host

struct SortPlan {
    int passes, tiles, blocks;
    bool one;
};
SortPlan sort_plan(const EmbedShape& s) {
    SortPlan p;
    p.passes = 1;
    while (p.passes < 4 && ((s.rows - 1) >> (p.passes * kDigit)) > 0) ++p.passes;
    p.one = s.tokens <= kOneBlock;
    const int64_t tiles = (s.tokens + kTile - 1) / kTile;
    p.tiles = int((tiles + kMaxBlocks - 1) / kMaxBlocks);
    p.blocks = int((tiles + p.tiles - 1) / p.tiles);
    return p;
}

// Vectors of channels: 16 bytes, or one value.
struct SumPlan {
    int v, x, y, slabs, piece;
    int64_t pieces;
};
// Pieces as long as they may be with some 64 warps on every SM: short ones write more partial sums, long ones leave SMs idle.  They
// decide in which order the sums are formed, so they depend on sizes and type alone: 152 SMs are reckoned with, and tensors on 16 bytes,
// whether they lie so or not.
SumPlan sum_plan(const EmbedShape& s, bool aligned) {
    const int size = s.dtype == UVU_F32 ? 4 : 2, v = s.inner == 1 && int64_t(s.channels) * size % 16 == 0 ? 16 / size : 1;
    SumPlan p;
    auto lay = [&](int width) {
        p.v = width;
        const int vecs = s.channels / p.v;
        p.x = 1;
        while (p.x < kSumThreads && p.x < vecs) p.x *= 2;
        p.y = kSumThreads / p.x;
        p.slabs = (vecs + p.x - 1) / p.x;
    };
    lay(v);
    const int64_t threads = int64_t(152) * 64 * 32, most = std::max<int64_t>(1, threads / (int64_t(p.x) * p.slabs));
    p.piece = kBatch;
    while (p.piece < 512 && (s.tokens + p.piece - 1) / p.piece > most) p.piece *= 2;
    p.pieces = (s.tokens + p.piece - 1) / p.piece;
    if (!aligned) lay(1);
    return p;
}

struct Work {
    uint32_t *keys[2], *counts, *totals;
    int32_t *ids[2], *valid, *chain;
    float* part;
    size_t bytes;
};
Work work_of(const EmbedShape& s, int64_t pieces, void* ws) {
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
        const bool needed = i == 0 || (!p.one && p.passes > 1);
        w.keys[i] = reinterpret_cast<uint32_t*>(take(needed ? size_t(s.tokens) * 4 : 0));
        w.ids[i] = reinterpret_cast<int32_t*>(take(needed ? size_t(s.tokens) * 4 : 0));
    }
    w.counts = reinterpret_cast<uint32_t*>(take(p.one ? 0 : size_t(p.blocks) * kBins * 4));
    w.totals = reinterpret_cast<uint32_t*>(take(kBins * 4));
    w.valid = reinterpret_cast<int32_t*>(take((kChains + kReaches) * sizeof(int32_t)));
    w.chain = reinterpret_cast<int32_t*>(take(size_t(pieces) * kReaches * 4));
    w.part = reinterpret_cast<float*>(take(size_t(pieces) * 2 * s.channels * 4));
    w.bytes = used;
    return w;
}

// Each kernel waits for the one before itself; the first of a call for all that came before.
template <typename... P, typename... Q>
cudaError_t launch(void (*k)(P...), dim3 grid, dim3 block, size_t smem, bool follows, cudaStream_t st, Q... args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = follows ? 1 : 0;
    return cudaLaunchKernelEx(&c, k, static_cast<P>(args)...);
}

template <typename T>
cudaError_t bwd(const EmbedShape& s, const int32_t* index, const void* dout, void* dtable, void* ws, int sms, cudaStream_t st) {
    const SortPlan p = sort_plan(s);
    const SumPlan m = sum_plan(s, ((reinterpret_cast<uintptr_t>(dout) | reinterpret_cast<uintptr_t>(dtable)) & 15u) == 0);
    const Work w = work_of(s, m.pieces, ws);
    unsigned char* table = static_cast<unsigned char*>(dtable);
    const int64_t bytes = s.rows * s.channels * int64_t(sizeof(T));
    const int zeros = int(std::min<int64_t>((bytes + 16383) / 16384, sms * 6));  // blocks that zero the table
    cudaError_t e = cudaSuccess;
    const uint32_t* keys = w.keys[0];
    const int32_t *ids = w.ids[0], *valid = w.valid;
    if (p.one) {
        e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOneSmem);
        const bool beside = bytes > kLargeTable;
        if (e == cudaSuccess)
            e = launch(sort_kernel, dim3(beside ? 1 : 1 + std::min(zeros, sms - 1)), dim3(kOneThreads), kOneSmem, false, st, int(s.tokens),
                       uint32_t(s.rows), p.passes, index, w.keys[0], w.ids[0], w.valid, table, bytes);
        if (e == cudaSuccess && beside) e = launch(zero_kernel, dim3(zeros), dim3(kThreads), 0, true, st, table, bytes);
    } else {
        Keys k = {s.tokens, uint32_t(s.rows), index, nullptr, nullptr, nullptr, 0, p.tiles};
        for (int i = 0; i < p.passes && e == cudaSuccess; ++i) {
            k.shift = i * kDigit;
            e = launch(count_kernel, dim3(p.blocks + (i == 0 ? zeros : 0)), dim3(kThreads), 0, i > 0, st, k, p.blocks, w.counts, table, bytes);
            if (e == cudaSuccess) e = launch(bins_kernel, dim3(kBins), dim3(kMaxBlocks), 0, true, st, p.blocks, w.counts, w.totals);
            if (e == cudaSuccess)
                e = launch(place_kernel, dim3(p.blocks), dim3(kThreads), 0, true, st, k, w.counts, w.totals, w.keys[i & 1], w.ids[i & 1],
                           w.valid, i & 1);
            k.keys = keys = w.keys[i & 1], k.ids = ids = w.ids[i & 1], k.valid = valid = w.valid + (i & 1);
        }
    }
    if (e != cudaSuccess) return e;
    const Sums u = {m.pieces, m.piece, s.channels, s.inner, s.column, float(s.scale), keys, ids, valid, w.part, w.valid + kChains, w.chain};
    const dim3 grid(unsigned((m.pieces + m.y - 1) / m.y), m.slabs), block(m.x, m.y);
    const T* d = static_cast<const T*>(dout);
    e = m.v == 1 ? launch(piece_kernel<T, 1>, grid, block, 0, true, st, u, d, static_cast<T*>(dtable))
                 : launch(piece_kernel<T, 16 / sizeof(T)>, grid, block, 0, true, st, u, d, static_cast<T*>(dtable));
    if (e != cudaSuccess || m.pieces < 2) return e;
    const int64_t most = std::min<int64_t>(m.pieces - 1, s.rows) * ((s.channels + 15) / 16);  // tasks
    return launch(join_kernel<T>, dim3(unsigned(std::min<int64_t>(most, sms * 8))), dim3(kJoinThreads), 0, true, st, u,
                  static_cast<T*>(dtable));
}

template <typename T>
cudaError_t fwd(const EmbedShape& s, const int32_t* index, const void* table, void* out, int sms, cudaStream_t st) {
    const int width = s.channels * s.inner;
    const bool plain = s.inner == 1;
    const uintptr_t any = reinterpret_cast<uintptr_t>(out) | uintptr_t(width) * sizeof(T) | (plain ? reinterpret_cast<uintptr_t>(table) : 0);
    auto go = [&](auto v, auto p) {
        constexpr int V = decltype(v)::value;
        constexpr bool P = decltype(p)::value;
        const int vecs = width / V;
        int x = 1;
        while (x < 256 && x < vecs) x *= 2;
        const int y = 256 / x;
        const int64_t blocks = (s.tokens + y * kLookupTokens - 1) / (y * kLookupTokens);
        const unsigned slabs = unsigned(std::min<int64_t>((vecs + x - 1) / x, std::max<int64_t>(1, int64_t(sms) * 8 / blocks)));
        embed_fwd_kernel<T, V, P><<<dim3(unsigned(blocks), slabs), dim3(x, y), 0, st>>>(
            s.tokens, uint32_t(s.rows), s.channels, s.inner, s.column, float(s.scale), index, static_cast<const T*>(table), static_cast<T*>(out));
        return cudaGetLastError();
    };
    auto by_inner = [&](auto v) { return plain ? go(v, std::true_type()) : go(v, std::false_type()); };
    if (any % 16 == 0) return by_inner(std::integral_constant<int, 16 / sizeof(T)>());
    if (sizeof(T) == 2 && any % 4 == 0) return by_inner(std::integral_constant<int, 4 / sizeof(T)>());
    return by_inner(std::integral_constant<int, 1>());
}

}  // namespace

size_t embed_workspace(const EmbedShape& s) {
    if (s.tokens == 0) return 0;
    return work_of(s, sum_plan(s, true).pieces, nullptr).bytes;
}

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
