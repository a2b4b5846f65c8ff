// Arguments of the attention kernels (attn.cu: launch choices and joining kernels).
#pragma once

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
    // split over the long axis: partial results, joined by a second kernel (splits == 1: none)
    int splits;
    float* part_o;    // forward [splits][nq][Hq][D]; backward: partial gradients
    float* part_lse;  // [splits][nq][Hq]
};

// Tile t of a packed batch whose graph b has (off[b+1] - off[b]) * per rows, R rows a tile:
// t(b) = off[b] * per / R + b is monotone in b and leaves every graph at least the tiles that it
// needs, so a grid of total * per / R + B tiles covers any batch; the spare numbers are empty.
struct AttnTile {
    int graph;     // -1: a spare number
    int64_t row0;  // first packed row, counted from the graph's first
    int64_t rows;  // packed rows of the graph
};
__device__ __forceinline__ AttnTile attn_tile(const int32_t* off, int graphs, int per, int R, int64_t t) {
    int lo = 0, hi = graphs;  // the last b with t(b) <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (int64_t(off[mid]) * per / R + mid <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int64_t a = off[lo], rows = (off[lo + 1] - a) * per;
    const int64_t r0 = (t - (a * per / R + lo)) * R;
    return {r0 < rows ? lo : -1, r0, rows};
}

// attn_mma.cu: the forward of 16-bit operands, nt (1 or 2) row tiles of 128 per block; a.splits > 1
// leaves partial results for the join.
cudaError_t launch_attn_fwd_mma(uvu_dtype dtype, const AttnArgs& a, int nt, int64_t row_tiles, cudaStream_t st);

// The backward of 16-bit operands: dk and dv (kv) by tiles of 128 states, or dq by tiles of 128 rows.
cudaError_t launch_attn_bwd_mma(uvu_dtype dtype, const AttnArgs& a, bool kv, int64_t tiles, cudaStream_t st);

// attn_planes.cu: fp32 operands as three bf16 planes each, in the workspace.  The backward's tiles have
// plane_bwd_tile() rows or states; above a head dimension of 64 it walks at most kPlaneWalk of the others in one piece.
constexpr int kPlaneWalk = 4096;
constexpr int plane_bwd_tile(int head_dim) { return head_dim <= 64 ? 128 : 64; }
size_t attn_planes_bytes(const AttnShape& s, bool bwd);
cudaError_t launch_attn_planes(const AttnArgs& a, void* ws, int sms, cudaStream_t st);
cudaError_t launch_attn_fwd_planes(const AttnArgs& a, void* ws, int64_t row_tiles, cudaStream_t st);
cudaError_t launch_attn_bwd_planes(const AttnArgs& a, void* ws, bool kv, int64_t tiles, cudaStream_t st);
// Status words of the files' kernels.
cudaError_t attn_fwd_mma_status(unsigned* word, bool reset);
cudaError_t attn_bwd_mma_status(unsigned* word, bool reset);
cudaError_t attn_planes_status(unsigned* word, bool reset);

}  // namespace uvu
