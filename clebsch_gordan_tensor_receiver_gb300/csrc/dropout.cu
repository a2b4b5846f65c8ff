// Dropout with an optional residual; the mask comes from a counter and is never stored.
//
//     y[e] = residual[e] + (keep(e / inner) ? x[e] * S : 0),   S = 65536 / (65536 - T),  T = round(65536 p)
//
// keep(d) compares 16 bits with T: draw d is half-word d % 8 (low half of each word first) of the
// Philox4x32-10 block with counter offset + d / 8 and the seed as key (Salmon, Moraes, Dror, Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  16 bits a draw make one block serve 8
// values: the ten rounds are some 80 instructions, and with 32-bit draws the 16-bit types would be
// bound by them instead of by memory.  S uses the probability that T stands for, so the expectation
// of y is exact although p is rounded to a multiple of 2^-16.  `inner` consecutive values share a
// draw: an equivariant feature keeps or loses all components of an irrep together.
//
// Bound by memory: x, residual and y move once.  A warp takes chunks of kSteps 16-byte vectors per
// lane: loads first, then the chunk's blocks (one per lane at a time, keep bits into shared
// memory), then the sums, so that the generator runs while the loads are on their way.  Measured: 262,144 x 512 in
// bf16, forward with residual and backward, 249 us (5390 GB/s of 1.34 GB; forward alone 62% issue, 58% of DRAM's rate);
// 1000 x 128 x 4 in fp32 3.5 us.
#include <algorithm>
#include <cstdint>

#include "elem.h"
#include "plan.h"

namespace uvu {
namespace {

constexpr int kThreads = 256, kSteps = 4;

// Keep bits of one block: bit i for draw i of the eight.
__device__ __forceinline__ uint32_t keep_bits(uint64_t counter, uint32_t k0, uint32_t k1, uint32_t limit) {
    uint32_t c0 = uint32_t(counter), c1 = uint32_t(counter >> 32), c2 = 0, c3 = 0;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = uint64_t(0xD2511F53u) * c0, b = uint64_t(0xCD9E8D57u) * c2;
        c0 = uint32_t(b >> 32) ^ c1 ^ (k0 + uint32_t(r) * 0x9E3779B9u);
        c2 = uint32_t(a >> 32) ^ c3 ^ (k1 + uint32_t(r) * 0xBB67AE85u);
        c1 = uint32_t(b);
        c3 = uint32_t(a);
    }
    const uint32_t w[4] = {c0, c1, c2, c3};
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bits |= uint32_t((w[i] & 0xFFFFu) >= limit) << (2 * i);
        bits |= uint32_t((w[i] >> 16) >= limit) << (2 * i + 1);
    }
    return bits;
}

// ONE: inner == 1 (a vector's draws are its own indices); RES: a residual is added.
template <typename T, int V, bool ONE, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(int64_t n, uint32_t inner, uint32_t k0, uint32_t k1, uint64_t offset,
                                                           uint32_t limit, float scale, const T* x,
                                                           const T* res, T* y) {
    constexpr int kChunk = kSteps * 32 * V;         // elements of a warp's chunk
    constexpr int kBlocks = kChunk / 8 + 2;         // Philox blocks that a chunk can touch
    __shared__ uint8_t s_keep[kThreads / 32][kBlocks];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* keep = s_keep[warp];
    const int64_t warps = int64_t(gridDim.x) * (kThreads / 32);
    for (int64_t base = (int64_t(blockIdx.x) * (kThreads / 32) + warp) * kChunk; base < n; base += warps * kChunk) {
        Vec<T, V> xv[kSteps], rv[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int64_t e = base + (s * 32 + lane) * V;
            if (e + V <= n) {
                xv[s] = load_vec<T, V>(x + e);
                if (RES) rv[s] = load_vec<T, V>(res + e);
            }
        }
        const int64_t d0 = ONE ? base : base / inner;  // first draw of the chunk
        const uint32_t r0 = ONE ? 0 : uint32_t(base - d0 * inner);
        const uint32_t first = uint32_t(d0 & 7);
        const uint32_t span = uint32_t(min(int64_t(kChunk), n - base)) - 1;
        const uint32_t blocks = (first + (ONE ? span : (r0 + span) / inner)) / 8 + 1;
        __syncwarp();  // the previous chunk's bits have been read
        for (uint32_t b = lane; b < blocks; b += 32)
            keep[b] = uint8_t(keep_bits(offset + uint64_t(d0 >> 3) + b, k0, k1, limit));
        __syncwarp();
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const uint32_t j = uint32_t(s * 32 + lane) * V;
            const int64_t e = base + j;
            if (e + V <= n) {
                Vec<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const uint32_t d = first + (ONE ? j + i : (r0 + j + i) / inner);
                    const bool on = (keep[d >> 3] >> (d & 7)) & 1;
                    const float t = on ? widen(xv[s].v[i]) * scale : 0.f;
                    o.v[i] = narrow<T>(RES ? widen(rv[s].v[i]) + t : t);
                }
                store_vec<T, V>(y + e, o);
            } else {
                for (int i = 0; i < V && e + i < n; ++i) {  // the last, partial vector
                    const uint32_t d = first + (ONE ? j + i : (r0 + j + i) / inner);
                    const bool on = (keep[d >> 3] >> (d & 7)) & 1;
                    const float t = on ? widen(x[e + i]) * scale : 0.f;
                    y[e + i] = narrow<T>(RES ? widen(res[e + i]) + t : t);
                }
            }
        }
    }
}

template <typename T, int V>
cudaError_t launch(int64_t n, int inner, uint32_t limit, uint64_t seed, uint64_t offset, const T* x, const T* res, T* y, int sms,
                   cudaStream_t st) {
    const float scale = limit < 65536 ? float(65536.0 / (65536.0 - limit)) : 0.f;
    const int64_t chunks = (n + kSteps * 32 * V - 1) / (kSteps * 32 * V);
    const int64_t blocks = (chunks + kThreads / 32 - 1) / (kThreads / 32);
    const unsigned grid = unsigned(std::min<int64_t>(blocks, int64_t(sms) * 8));
    const uint32_t k0 = uint32_t(seed), k1 = uint32_t(seed >> 32);
    auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, st>>>(n, uint32_t(inner), k0, k1, offset, limit, scale, x, res, y); };
    if (inner == 1)
        res ? go(dropout_kernel<T, V, true, true>) : go(dropout_kernel<T, V, true, false>);
    else
        res ? go(dropout_kernel<T, V, false, true>) : go(dropout_kernel<T, V, false, false>);
    return cudaGetLastError();
}

template <typename T>
cudaError_t by_alignment(int64_t n, int inner, uint32_t limit, uint64_t seed, uint64_t offset, const void* x, const void* res,
                         void* y, int sms, cudaStream_t st) {
    const T *xp = static_cast<const T*>(x), *rp = static_cast<const T*>(res);
    T* yp = static_cast<T*>(y);
    const uintptr_t any = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(res) | reinterpret_cast<uintptr_t>(y);
    // 16-byte vectors need 16-byte aligned tensors; a view that begins elsewhere goes element by element
    return any & 15u ? launch<T, 1>(n, inner, limit, seed, offset, xp, rp, yp, sms, st)
                     : launch<T, 16 / sizeof(T)>(n, inner, limit, seed, offset, xp, rp, yp, sms, st);
}

}  // namespace

cudaError_t launch_dropout(uvu_dtype dtype, int64_t n, int inner, uint32_t limit, uint64_t seed, uint64_t offset, const void* x,
                           const void* residual, void* y, int sms, cudaStream_t st) {
    switch (dtype) {
        case UVU_F32: return by_alignment<float>(n, inner, limit, seed, offset, x, residual, y, sms, st);
        case UVU_BF16: return by_alignment<__nv_bfloat16>(n, inner, limit, seed, offset, x, residual, y, sms, st);
        case UVU_F16: return by_alignment<__half>(n, inner, limit, seed, offset, x, residual, y, sms, st);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace uvu
