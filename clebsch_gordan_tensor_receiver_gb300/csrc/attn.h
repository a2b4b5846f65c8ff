// Arguments of the attention kernels (attn.cu: launch choices and joining kernels).
#pragma once

#include <algorithm>

#include "plan.h"

namespace uvu {

// One call.  Rows are packed: for graph b and kv head h the query rows are r = i * group + j (query i
// of the graph, head h * group + j), so that the heads that share K and V share tiles too.
struct AttnArgs {
    int graphs, Hq, Hkv, group, D;
    int64_t nq, nk;           // rows of all graphs
    float scale, scale_log2;  // scale, scale * log2(e)
    int64_t q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;  // strides in elements
    const int32_t *q_off, *k_off;
    const uint8_t* keep;  // [nk] or null
    const void *q, *k, *v;
    void* out;
    float* lse;  // [nq][Hq]
    // backward
    const void* d_out;
    void *dq, *dk, *dv;  // contiguous
    float* delta;        // [nq][Hq]: sum_d d_out out
    // f16 operands: what the scale of dS follows (attn_mma_bwd.cu)
    float *do2, *v2;             // [nq][Hq]: sum_d d_out^2; [nk][Hkv]: sum_d v^2 of kept states, else 0
    unsigned *do2_top, *v2_top;  // [graphs][Hkv]: their maxima over a graph's rows and the kv head's heads, as bits
    // split over the long axis: partial results, joined by a second kernel (1: none)
    int splits;
    float* part_o;    // [splits][nq][Hq][D]; of one walk too where it is held
    bool hold;        // walks are long (attn_hold_tiles); in the backward some of them
    float* part_lse;  // [splits][nq][Hq]
    // backward
    int64_t kv_tiles, q_tiles;  // tile numbers of dk and dv, and of dq (0: not asked for)
    bool q_first;
    int splits_kv, splits_q;
    // [2][splits_kv][nk][Hkv][D], [splits_q][nq][Hq][D]; null: one walk, which is not held
    float *part_kv, *part_q;
};

// Tile t of a packed batch whose graph b has (off[b+1] - off[b]) * per rows, R rows a tile:
// t(b) = off[b] * per / R + b is monotone in b and leaves every graph at least the tiles that it
// needs, so a grid of total * per / R + B tiles covers any batch; the spare numbers are empty.
struct AttnTile {
    int graph;            // -1: a spare number
    int64_t row0, rows;   // first packed row of the tile, and packed rows of the graph
    int64_t first;        // the graph's first row
    int64_t other, n;     // the first row and the rows of the graph on the other side
};
// By all threads of the block (it synchronises them).  One round of loads finds the graph of a moderate batch,
// each thread testing some; a large one is searched by halves first.
template <int R>
__device__ __forceinline__ AttnTile attn_tile(const int32_t* off, const int32_t* other, int graphs, int per, int64_t t) {
    __shared__ int s[5];
    int lo = 0, hi = graphs;  // the last b with t(b) <= t is in [lo, hi)
    while (hi - lo > 4 * int(blockDim.x)) {
        const int mid = (lo + hi) >> 1;
        if (int64_t(off[mid]) * per / R + mid <= t)
            lo = mid;
        else
            hi = mid;
    }
    for (int b = lo + int(threadIdx.x); b < hi; b += int(blockDim.x)) {
        const int x = off[b], y = off[b + 1], u = other[b], v = other[b + 1];
        if (int64_t(x) * per / R + b <= t && (b + 1 == graphs || t < int64_t(y) * per / R + b + 1))
            s[0] = b, s[1] = x, s[2] = y, s[3] = u, s[4] = v;
    }
    __syncthreads();
    AttnTile r;
    r.first = s[1], r.rows = int64_t(s[2] - s[1]) * per, r.other = s[3], r.n = s[4] - s[3];
    r.row0 = (t - (int64_t(s[1]) * per / R + s[0])) * R;
    r.graph = r.row0 < r.rows ? s[0] : -1;
    return r;
}

// Tiles of 128 states or rows whose products one sum in tensor memory takes.  Each accumulating instruction (16 states) cuts the
// sum by up to 2^-23 of it: values of one sign lose 1.1e-4 over 16384 states, a fifth of f16's u, and 4e-4 over 65536, a tenth
// of bf16's.  Longer walks add such sums up in fp32 in memory; without that, 2^20 states were off by 6.7e-3 in f16.
__host__ __device__ constexpr int attn_hold_tiles(bool f16) { return f16 ? 128 : 512; }

// attn_mma.cu: the forward of 16-bit operands, nt (1 or 2) row tiles of 128 per block; a.splits > 1
// leaves partial results for the join.
cudaError_t launch_attn_fwd_mma(uvu_dtype dtype, const AttnArgs& a, int nt, int64_t row_tiles, cudaStream_t st);

// One launch for dk, dv and dq.  The kind whose tiles walk further comes first, for all heads, so that the short ones
// fill the end (a tile of dk and dv walks the rows, one of dq the states): 16 heads of 128, 4 x 4096 rows and states
// 2.34 -> 2.24 ms in bf16, against heads in the order of the grid, each with its dk and dv first.
struct BwdTile {
    bool kv;
    int head;
    int64_t tile;
};
__device__ __forceinline__ BwdTile bwd_tile_of(const AttnArgs& a) {
    const int64_t n = blockIdx.x / unsigned(a.Hkv), first = a.q_first ? a.q_tiles : a.kv_tiles;
    return {(n < first) != a.q_first, int(blockIdx.x % unsigned(a.Hkv)), n < first ? n : n - first};
}
inline dim3 bwd_grid(const AttnArgs& a) {
    return dim3(unsigned((a.kv_tiles + a.q_tiles) * a.Hkv), 1, unsigned(std::max(a.splits_kv, a.splits_q)));
}

// The backward of 16-bit operands in tiles of 128 states or rows.
cudaError_t launch_attn_bwd_mma(uvu_dtype dtype, const AttnArgs& a, cudaStream_t st);

// attn_planes.cu: fp32 operands as three bf16 planes each, in the workspace.  The backward's tiles have
// plane_bwd_tile() rows or states.
constexpr int plane_bwd_tile(int head_dim) { return head_dim <= 64 ? 128 : 64; }
size_t attn_planes_bytes(const AttnShape& s, bool bwd);
// Writes the planes of q, k and v; for the backward those of d_out too, and delta.
cudaError_t launch_attn_planes(const AttnArgs& a, void* ws, int sms, cudaStream_t st);
cudaError_t launch_attn_fwd_planes(const AttnArgs& a, void* ws, int64_t row_tiles, cudaStream_t st);
cudaError_t launch_attn_bwd_planes(const AttnArgs& a, void* ws, cudaStream_t st);
// Status words of the files' kernels.
cudaError_t attn_fwd_mma_status(unsigned* word, bool reset);
cudaError_t attn_bwd_mma_status(unsigned* word, bool reset);
cudaError_t attn_planes_status(unsigned* word, bool reset);

}  // namespace uvu
