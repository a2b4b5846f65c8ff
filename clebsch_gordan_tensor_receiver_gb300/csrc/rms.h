// What the kernels of the RMS norm share (rms_fwd.cu, rms_quant.cu, rms_bwd.cu; rows of more than 8192 values: rms_wide.cu).
//
//     h = round(x + residual),  r = (mean h^2 + eps)^(-1/2),  y = h r gamma          (a row: channels * inner values)
//     8 bits, for each group of a row:  s = max |y| / 448,  q = e4m3(y / s)
//     d_x = d_h + r (t - u mean(t u)),  t = gamma d_y,  u = h r;   d_gamma[c] = sum over rows and components of d_y u
//
// gamma is one value a channel, shared by the `inner` components of an irrep, so y is as equivariant as x.  The norm is of h as
// it is stored: what the next layer and the gradient read is what was normalised.
//
// Bound by memory: every tensor moves once. A row belongs to a team, a part of a warp or a block, whose threads hold it in registers, 16
// values each at most, between the sum and the result. The team's next rows are on their way to shared memory meanwhile, by asynchronous
// copies that cost no registers: with one row ahead in registers the gradient had 48 KB in flight on an SM and ran at half of the memory's
// rate. Rows that do not begin on 16 bytes are read in words, one row ahead in registers (copied in whole chunks, with what lies before and
// behind them, they took twice the time), also where every other one begins inside a word. 262,144 x 512 in bf16 with the residual: 341 us
// forward and back (6.3 TB/s); 65,537 x 1024 to 8 bits 88 us (5.4 TB/s); 96,064 x 427 in f16 with the residual: 63 us (5.2 TB/s) forward,
// 90 us (3.7 TB/s) back, to 8 bits 71 us (4.0 TB/s), with groups of 64, which lanes do not share evenly, 172 us. A thread has the same
// columns of every row that it sees, so gamma is read once, and d_gamma is summed in registers, then over the block's teams in shared
// memory, and over the blocks, in their order, by a second kernel.
#pragma once

#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "elem.h"
#include "plan.h"
#include "tensor_core.h"

namespace uvu {
namespace {

enum RmsMode { kRmsFwd, kRmsQuant, kRmsQuantAny, kRmsBwd };  // Any: groups that lanes do not share evenly
// How a row ends: kCut, inside a step or where one ends; kFull, where the steps end; kOdd, 16-bit rows of odd length, see RmsRow
enum RmsEnd { kCut, kFull, kOdd };

constexpr int kTeamRows = 512;      // rows that a team adds up in one fp32 sum of d_gamma
constexpr int kValues = 16;         // of a thread, at most
constexpr int kAhead = 3;           // rows on their way, beside the one at work; one where shared memory does not hold three
constexpr size_t kRowsSmem = 200 << 10;
constexpr float kTop = 448.f;       // the largest e4m3 value

template <int V>
struct alignas(V) Bytes {
    uint8_t b[V];
    __device__ __forceinline__ void set(const float* v) {
        if constexpr (V == 1) {
            b[0] = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
        } else {
            uint16_t w[(V + 1) / 2];
#pragma unroll
            for (int i = 0; i < (V + 1) / 2; ++i) w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            __builtin_memcpy(b, w, sizeof(w));
        }
    }
};

// A NaN is kept.
__device__ __forceinline__ float nan_max(float a, float b) {
    float c;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
    return c;
}
__device__ __forceinline__ float inv_sqrt(float v) {  // of what is not subnormal
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// Of a mean of squares that eps is added to: whether squares may have left fp32, or may lie below it where eps does not hide them.  One
// comparison of the bits: not 2^-80 <= mean < 2^126.
__device__ __forceinline__ bool squares_beyond(float mean) { return __float_as_uint(mean) - 0x17800000u >= 0x7E800000u - 0x17800000u; }
// The values' factor for another try.
__device__ __forceinline__ float squares_factor(float mean) { return mean < 1.f ? 0x1p90f : 0x1p-80f; }

// A group's scale, s = top / 448 of its largest |y|, and its values divided by it: quotients in fp32, of which the 8 bits are formed (a
// product with the inverse can fall on the other side of the middle between two e4m3 values).  Zeros stay zeros, a NaN makes all NaN.
//
// Where nothing leaves fp32's range, by a quotient's last step (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990): q = v f with f = 1/s to some 2^-23, then q + (v - q s) f, whose error before it is rounded is 2^-44.
// As divisions: 114 us for 65,537 x 1024 from bf16.  Whether a scale is too small or large for it is asked once a row, by a
// whole warp: a branch for each vector made 96,064 x 428 take 88 us where this takes 60.
struct Scale {
    float s, f;  // f: NaN where fp32's range may be left; 0 for zeros
    __device__ __forceinline__ Scale() {}
    __device__ __forceinline__ Scale(float scale, float inverse) : s(scale), f(inverse) {}
    __device__ __forceinline__ explicit Scale(float top) {
        const float q = top * (1.f / kTop);
        s = fmaf(fmaf(-q, kTop, top), 1.f / kTop, q);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"(s));
        // not 2^-70 <= top < 2^108, by one comparison of the bits (a remainder that fp32 does not hold is of a value that rounds to zero)
        if (__builtin_expect(__float_as_uint(top) - 0x1C800000u >= 0x75800000u - 0x1C800000u, 0)) {
            s = top / kTop;
            f = s == 0.f ? 0.f : NAN;
        }
    }
    __device__ __forceinline__ bool rare() const { return f != f; }
    template <bool RARE, int N>
    __device__ __forceinline__ void divide(const float* v, float (&u)[N]) const {
        if constexpr (RARE) {
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = s == 0.f ? 0.f : v[i] / s;
        } else {
#pragma unroll
            for (int i = 0; i + 1 < N; i += 2) {
                const F2 w(v[i], v[i + 1]), q = w * F2(f, f);
                const float2 r = fma2(fma2(q, F2(-s, -s), w), F2(f, f), q).both();
                u[i] = r.x, u[i + 1] = r.y;
            }
            if constexpr (N % 2 == 1) {
                const float q = v[N - 1] * f;
                u[N - 1] = fmaf(fmaf(q, -s, v[N - 1]), f, q);
            }
        }
    }
};

struct RmsArgs {
    int64_t rows;
    int width, inner, team;        // width: values of a row
    int group, groups;             // values that share a scale, and scales of a row
    float eps;
    const void* in[3];             // x, residual; gradient: h, dy, dh (residual, dh: or NULL)
    void* out[2];                  // y, h (NULL without a residual); gradient: dx
    const float* gamma;
    float *rstd, *scales, *partial;
    int64_t block_rows;            // of the gradient
    int ahead;                     // kAhead or 1
    int n_in, slot;                // inputs that are there, and bytes of a row's place in shared memory
};

// ------------------------------------------------------------------------------------ one row

// V consecutive columns a thread and step, K steps; WARP: the team is a power of two of lanes, else the block.
//
// kOdd: every other row begins between two words.  A team's rows are an even number apart, so they all do or all do not: its words are
// those of columns 0, 1, .. or 1, 2, .., and the single column left, the last one or the first, is the first lane's.
template <typename T, int V, int K, bool WARP, RmsEnd END, RmsMode MODE>
struct RmsRow {
    static constexpr int kLone = END == kOdd ? 1 : 0, kN = K * V;  // the single column's value stands behind the others
    template <int W>  // (whole rows, which no condition stands before, were 7% faster to 8 bits as single values)
    using Values = Pack<T, W, END != kFull>;
    float gamma[kN + kLone];
    float acc[MODE == kRmsBwd ? kN + kLone : 1];
    int lane, team, width, from, lone;
    bool has_lone;
    float inv, eps;

    __device__ __forceinline__ RmsRow(const RmsArgs& a, int64_t row) {
        team = WARP ? a.team : int(blockDim.x);
        lane = WARP ? int(threadIdx.x) & (team - 1) : int(threadIdx.x);
        width = a.width;
        from = END == kOdd ? int(row & 1) : 0;
        lone = from ? 0 : width - 1;
        has_lone = END == kOdd && lane == 0;
        inv = 1.f / float(width);
        eps = a.eps;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = column(k) + i;
                gamma[k * V + i] = inside(k) && e < width ? a.gamma[e / a.inner] : 0.f;
                if (MODE == kRmsBwd) acc[k * V + i] = 0.f;
            }
        if constexpr (END == kOdd) {
            gamma[kN] = has_lone ? a.gamma[lone / a.inner] : 0.f;
            if (MODE == kRmsBwd) acc[kN] = 0.f;
        }
    }
    __device__ __forceinline__ int column(int k) const { return from + (k * team + lane) * V; }
    __device__ __forceinline__ bool inside(int k) const { return END == kFull || (k * team + lane) * V < width - kLone; }

    // Over the team, in all of its threads.  s_part: another half from row to row, so that the last sum has been read.
    __device__ __forceinline__ float sum(float v, float* s_part) const {
        if (WARP) {
            for (int d = team >> 1; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
            return v;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
        for (int w = 0; w < team >> 5; ++w) v += s_part[w];
        return v;
    }
    __device__ __forceinline__ void sync() const {
        if (WARP) __syncwarp();
        else __syncthreads();
    }

    // Rows that begin on 16 bytes have places in shared memory, [ahead + 1][n_in][slot] bytes for each team; a thread copies there what
    // it will read.
    static constexpr bool kWhole = V * sizeof(T) == 16;
    static constexpr int kIn = MODE == kRmsBwd ? 3 : 2;

    // `at`: of the row's first value
    __device__ __forceinline__ void fetch(const RmsArgs& a, int64_t at, bool live, uint32_t to) const {
#pragma unroll
        for (int j = 0; j < kIn; ++j)
            if (live && j < a.n_in) {
                const T* p = static_cast<const T*>(a.in[j]) + at;
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (inside(k)) tc::copy16(to + j * a.slot + column(k) * int(sizeof(T)), p + column(k), 16);
            }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // The row that was asked for longest ago is there.
    __device__ __forceinline__ void arrived(int ahead) const {
        if (ahead == kAhead) asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
        else asm volatile("cp.async.wait_group 1;" ::: "memory");
    }
    struct Read {
        Values<V> t[kIn][K];
        Values<1> lone[kIn];  // kOdd
        float r;
    };
    // From shared memory (places a.slot bytes apart), or from the tensors.
    template <bool STAGED>
    __device__ __forceinline__ void take(const RmsArgs& a, int64_t at, bool live, const unsigned char* from, Read& in) const {
#pragma unroll
        for (int j = 0; j < kIn; ++j) {
            const bool there = live && j < a.n_in;
            const T* p = STAGED ? reinterpret_cast<const T*>(from + j * a.slot) : static_cast<const T*>(a.in[j]) + at;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (there && inside(k)) in.t[j][k] = *reinterpret_cast<const Values<V>*>(p + column(k));
                else in.t[j][k].clear();
            }
            if constexpr (END == kOdd) {
                if (there && has_lone) in.lone[j] = *reinterpret_cast<const Values<1>*>(p + lone);
                else in.lone[j].clear();
            }
        }
    }

    // The values of h in v and its 1 / sqrt(mean h^2 + eps); h is written where there is a residual.
    template <int W>
    __device__ __forceinline__ static void add(const Values<W>& x, const Values<W>& r, bool res, T* h, int column, bool write, float* v, float& s) {
        x.get(v);
        if (res) {
            float u[W];
            r.get(u);
#pragma unroll
            for (int i = 0; i < W; ++i) u[i] += v[i];
            Values<W> o;
            o.set(u);
            o.get(v);
            if (write) *reinterpret_cast<Values<W>*>(h + column) = o;
        }
#pragma unroll
        for (int i = 0; i < W; ++i) s = fmaf(v[i], v[i], s);
    }
    __device__ __forceinline__ float load(const Read& in, bool res, T* h, bool live, float* s_part, float (&v)[kN + kLone]) const {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) add(in.t[0][k], in.t[1][k], res, h, column(k), live && inside(k), v + k * V, s);
        if constexpr (END == kOdd) add(in.lone[0], in.lone[1], res, h, lone, live && has_lone, v + kN, s);
        const float mean = fmaf(sum(s, s_part), inv, eps);
        float r = inv_sqrt(mean);
        // rarely, and then once more at another scale (all lanes of a warp take part in its teams' sums)
        const bool beyond = squares_beyond(mean);
        if (__builtin_expect(WARP ? __any_sync(0xffffffffu, beyond) : beyond, 0)) {
            const float f = squares_factor(mean);
            s = 0.f;
#pragma unroll
            for (int i = 0; i < kN + kLone; ++i) s = fmaf(v[i] * f, v[i] * f, s);
            if (!WARP) __syncthreads();  // the first sums have been read
            s = sum(s, s_part);
            if (beyond) r = inv_sqrt(fmaf(s, inv, eps * f * f)) * f;
        }
        return r;
    }

    template <int W>
    __device__ __forceinline__ static void scale(const float* v, const float* gamma, float r, T* y) {
        float u[W];
#pragma unroll
        for (int i = 0; i < W; ++i) u[i] = v[i] * r * gamma[i];
        Values<W> o;
        o.set(u);
        *reinterpret_cast<Values<W>*>(y) = o;
    }
    __device__ __forceinline__ void forward(const Read& in, bool res, T* y, T* h, float* rstd, bool live, float* s_part) const {
        float v[kN + kLone];
        const float r = load(in, res, h, live, s_part, v);
        if (live && lane == 0 && rstd) *rstd = r;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (live && inside(k)) scale<V>(v + k * V, gamma + k * V, r, y + column(k));
        if constexpr (END == kOdd)
            if (live && has_lone) scale<1>(v + kN, gamma + kN, r, y + lone);
    }

    // s_top (kRmsQuantAny): two words for each group of the row.
    __device__ __forceinline__ void quantise(const Read& in, bool res, uint8_t* q, T* h, float* scales, int group, int groups, bool live,
                                             float* s_part, unsigned* s_top) const {
        float v[kN + kLone];
        const float r = load(in, res, h, live, s_part, v);
        float top[K];
        if constexpr (END == kOdd) v[kN] = v[kN] * r * gamma[kN];  // in the forward's order: its y
#pragma unroll
        for (int k = 0; k < K; ++k) {
            top[k] = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[k * V + i] = v[k * V + i] * r * gamma[k * V + i];
                top[k] = nan_max(top[k], fabsf(v[k * V + i]));
            }
        }
        if constexpr (MODE == kRmsQuantAny) {
            sync();  // the last row's have been read
            for (int j = lane; j < groups; j += team) s_top[j] = 0u;
            sync();
            const bool by_warp = END != kOdd && team >= 32 && group % (32 * V) == 0;  // the lanes of a step share a group
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = column(k), g = c / group;
                if (by_warp) {
                    const unsigned most = __reduce_max_sync(0xffffffffu, live && inside(k) ? __float_as_uint(top[k]) : 0u);
                    if ((threadIdx.x & 31) == 0 && g < groups) atomicMax(s_top + g, most);
                } else if (live && inside(k)) {
                    if ((c + V - 1) / group == g) {
                        atomicMax(s_top + g, __float_as_uint(top[k]));
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) atomicMax(s_top + (c + i) / group, __float_as_uint(fabsf(v[k * V + i])));
                    }
                }
            }
            if constexpr (END == kOdd)
                if (live && has_lone) atomicMax(s_top + lone / group, __float_as_uint(fabsf(v[kN])));
            sync();
            float *s_scale = reinterpret_cast<float*>(s_top), *s_inverse = s_scale + groups;
            bool rare = false;
            for (int j = lane; j < groups; j += team) {
                const Scale scale(__uint_as_float(s_top[j]));
                s_scale[j] = scale.s, s_inverse[j] = scale.f;
                if (live) scales[j] = scale.s;
                rare |= scale.rare();
            }
            if (WARP) __syncwarp();
            else rare = __syncthreads_or(rare);
            auto scale_of = [&](int g) { return Scale(s_scale[g], s_inverse[g]); };
            auto give = [&](auto rare) {
                constexpr bool RARE = decltype(rare)::value;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int c = column(k), g = c / group;
                    if (!live || !inside(k)) continue;
                    float u[V];
                    if ((c + V - 1) / group == g) {
                        scale_of(g).template divide<RARE>(v + k * V, u);
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            float one[1];
                            scale_of((c + i) / group).template divide<RARE>(v + k * V + i, one);
                            u[i] = one[0];
                        }
                    }
                    Bytes<V> o;
                    o.set(u);
                    *reinterpret_cast<Bytes<V>*>(q + c) = o;
                }
                if constexpr (END == kOdd)
                    if (live && has_lone) give_lone<RARE>(scale_of(lone / group), v + kN, q);
            };
            if (__builtin_expect(__any_sync(0xffffffffu, rare), 0)) give(std::true_type());
            else give(std::false_type());
        } else {
            // The largest |y| of a thread's group, for each step.  A group is the row, a power of two of a step's lanes, or a power of two
            // of a warp's whole steps.
            const bool whole = group >= width;
            const int lanes = group / V, bits = 31 - __clz(group);
            if (whole) {
                float t = top[0];
#pragma unroll
                for (int k = 1; k < K; ++k) t = nan_max(t, top[k]);
                if constexpr (END == kOdd) t = nan_max(t, fabsf(v[kN]));
                for (int d = min(team, 32) >> 1; d > 0; d >>= 1) t = nan_max(t, __shfl_xor_sync(0xffffffffu, t, d));
                if (!WARP) {
                    float* s_max = s_part + 32;
                    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = t;
                    __syncthreads();
                    for (int w = 0; w < team >> 5; ++w) t = nan_max(t, s_max[w]);
                }
                top[0] = t;
            } else {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    for (int d = min(lanes, 32) >> 1; d > 0; d >>= 1) top[k] = nan_max(top[k], __shfl_xor_sync(0xffffffffu, top[k], d));
#pragma unroll
                for (int d = 1; d < K; d *= 2)
                    if (32 * d < lanes) {
                        float other[K];
#pragma unroll
                        for (int k = 0; k < K; ++k) other[k] = (k ^ d) < K ? top[(k ^ d) < K ? k ^ d : k] : 0.f;
#pragma unroll
                        for (int k = 0; k < K; ++k) top[k] = nan_max(top[k], other[k]);
                    }
            }
            // one group: `whole`, and rows of odd length (others of those are kRmsQuantAny's)
            auto give = [&](auto rare, auto scale) {
                constexpr bool RARE = decltype(rare)::value;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int c = column(k);
                    if (!live || !inside(k)) continue;
                    float u[V];
                    scale(k).template divide<RARE>(v + k * V, u);
                    if (whole ? k == 0 && lane == 0 : (c & (group - 1)) == 0) scales[whole ? 0 : c >> bits] = scale(k).s;
                    Bytes<V> o;
                    o.set(u);
                    *reinterpret_cast<Bytes<V>*>(q + c) = o;
                }
                if constexpr (END == kOdd)
                    if (live && has_lone) give_lone<RARE>(scale(0), v + kN, q);
            };
            auto give_either = [&](bool rare, auto scale) {
                if (__builtin_expect(__any_sync(0xffffffffu, rare), 0)) give(std::true_type(), scale);
                else give(std::false_type(), scale);
            };
            if (whole) {
                const Scale one(top[0]);
                give_either(one.rare(), [&](int) { return one; });
            } else if constexpr (END != kOdd) {
                Scale each[K];
                bool rare = false;
#pragma unroll
                for (int k = 0; k < K; ++k) each[k] = Scale(top[k]), rare |= each[k].rare();
                give_either(rare, [&](int k) { return each[k]; });
            }
        }
    }
    template <bool RARE>
    __device__ __forceinline__ void give_lone(const Scale& scale, const float* v, uint8_t* q) const {
        float u[1];
        scale.template divide<RARE>(v, u);
        Bytes<1> o;
        o.set(u);
        q[lone] = o.b[0];
    }

    // d_gamma += d_y u, and the sum of gamma d_y u
    template <int W>
    __device__ __forceinline__ static void gather(const Values<W>& xv, const Values<W>& gv, const float* gamma, float r, float* acc, float& dot) {
        float x[W], g[W];
        xv.get(x);
        gv.get(g);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const float u = x[i] * r;
            acc[i] = fmaf(g[i], u, acc[i]);
            dot = fmaf(g[i] * gamma[i], u, dot);
        }
    }
    template <int W>
    __device__ __forceinline__ static void give(const Values<W>& xv, const Values<W>& gv, const Values<W>& hv, const float* gamma, float r,
                                                float mean, T* dx) {
        float x[W], g[W], t[W];
        xv.get(x);
        gv.get(g);
        hv.get(t);
#pragma unroll
        for (int i = 0; i < W; ++i) t[i] = fmaf(fmaf(-x[i] * r, mean, g[i] * gamma[i]), r, t[i]);  // r r may be beyond fp32
        Values<W> o;
        o.set(t);
        *reinterpret_cast<Values<W>*>(dx) = o;
    }
    __device__ __forceinline__ void backward(const Read& in, T* dx, bool live, float* s_part) {
        const float r = in.r;
        constexpr int kDh = MODE == kRmsBwd ? 2 : 0;
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) gather(in.t[0][k], in.t[1][k], gamma + k * V, r, acc + k * V, dot);
        if constexpr (END == kOdd) gather(in.lone[0], in.lone[1], gamma + kN, r, acc + kN, dot);
        const float mean = sum(dot, s_part) * inv;  // of t u
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (live && inside(k)) give(in.t[0][k], in.t[1][k], in.t[kDh][k], gamma + k * V, r, mean, dx + column(k));
        if constexpr (END == kOdd)
            if (live && has_lone) give(in.lone[0], in.lone[1], in.lone[kDh], gamma + kN, r, mean, dx + lone);
    }

    // The block's sums of d_gamma, over its teams and a channel's components in their order.  s_sum [teams][width]
    __device__ __forceinline__ void give_gradient(const RmsArgs& a, float* s_sum) const {
        const int teams = WARP ? int(blockDim.x) / team : 1, mine = WARP ? int(threadIdx.x) / team : 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (inside(k) && column(k) + i < width) s_sum[mine * width + column(k) + i] = acc[k * V + i];
        if constexpr (END == kOdd)
            if (has_lone) s_sum[mine * width + lone] = acc[kN];
        __syncthreads();
        const int channels = width / a.inner;
        for (int c = threadIdx.x; c < channels; c += blockDim.x) {
            float s = 0.f;
            for (int i = 0; i < a.inner; ++i)
#pragma unroll 4
                for (int m = 0; m < teams; ++m) s += s_sum[m * width + c * a.inner + i];
            a.partial[int64_t(blockIdx.x) * channels + c] = s;
        }
    }
};

// ----------------------------------------------------------------------------------- the kernel

template <typename T, int V, int K, bool WARP, RmsEnd END, RmsMode MODE>
__global__ void __launch_bounds__(WARP ? 256 : V == 1 ? 1024 : 512) rms_kernel(const RmsArgs a) {
    __shared__ float s_part[2][64];
    // the rows' places, then the groups' maxima; at the end the sums of d_gamma
    extern __shared__ __align__(16) unsigned char smem[];
    if (MODE == kRmsBwd) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join begins as blocks end
    using Row = RmsRow<T, V, K, WARP, END, MODE>;
    const int teams = WARP ? int(blockDim.x) / a.team : 1, mine = WARP ? int(threadIdx.x) / a.team : 0;
    T* out1 = static_cast<T*>(a.out[1]);
    unsigned* s_top = reinterpret_cast<unsigned*>(smem + teams * (a.ahead + 1) * a.n_in * a.slot);
    // The gradient's rows of a block lie together, so that its sums are of rows in their order; not those of whole blocks and odd length,
    // whose rows would not be an even number apart.
    constexpr bool kTogether = MODE == kRmsBwd && (WARP || END != kOdd);
    const int64_t step = kTogether ? teams : int64_t(gridDim.x) * teams;
    const int64_t first = kTogether ? blockIdx.x * a.block_rows : int64_t(blockIdx.x) * teams;
    const int64_t end = kTogether ? min(first + a.block_rows, a.rows) : a.rows;
    Row op(a, first + mine);
    typename Row::Read now;
    const int64_t stride = step * a.width;  // values between a team's rows
    int half = 0;
    auto work = [&](int64_t row, int64_t at, bool live) {
        if constexpr (MODE == kRmsFwd)
            op.forward(now, out1 != nullptr, static_cast<T*>(a.out[0]) + at, out1 + at, a.rstd ? a.rstd + row : nullptr, live, s_part[half]);
        else if constexpr (MODE == kRmsQuant || MODE == kRmsQuantAny)
            op.quantise(now, out1 != nullptr, static_cast<uint8_t*>(a.out[0]) + at, out1 + at, a.scales + row * a.groups, a.group, a.groups,
                        live, s_part[half], s_top + mine * 2 * a.groups);
        else
            op.backward(now, static_cast<T*>(a.out[0]) + at, live, s_part[half]);
        half ^= 1;
    };
    auto rstd_of = [&](int64_t row) { return MODE == kRmsBwd && row < end ? a.rstd[row] : 0.f; };
    if constexpr (Row::kWhole) {
        const int places = a.n_in * a.slot;  // bytes of a row's
        unsigned char* ring = smem + mine * (a.ahead + 1) * places;
        const uint32_t ring_at = tc::smem_u32(ring);
        float r[MODE == kRmsBwd ? kAhead : 1] = {};  // rstd of the rows on their way
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i < a.ahead) {
                const int64_t row = first + mine + i * step;
                op.fetch(a, row * a.width, row < end, ring_at + i * places);
                if constexpr (MODE == kRmsBwd) r[i] = rstd_of(row);
            }
        int place = 0, free = a.ahead;
        int64_t row = first + mine, at = row * a.width;
        const int64_t rows_ahead = a.ahead * step, values_ahead = a.ahead * stride;
        for (int64_t base = first; base < end; base += step, row += step, at += stride) {
            op.fetch(a, at + values_ahead, row + rows_ahead < end, ring_at + free * places);
            op.arrived(a.ahead);
            op.template take<true>(a, at, row < end, ring + place * places, now);
            if constexpr (MODE == kRmsBwd) {
                const float last = rstd_of(row + rows_ahead);
                now.r = r[0];
#pragma unroll
                for (int i = 0; i + 1 < kAhead; ++i) r[i] = r[i + 1];
                r[kAhead - 1] = last;
                if (a.ahead == 1) r[0] = last;
            }
            work(row, at, row < end);
            free = place;
            place = place == a.ahead ? 0 : place + 1;
        }
        tc::copy_wait_all();
    } else {
        typename Row::Read next;
        auto ask = [&](int64_t row, int64_t at) {
            op.template take<false>(a, at, row < end, nullptr, next);
            next.r = rstd_of(row);
        };
        int64_t row = first + mine, at = row * a.width;
        ask(row, at);
        for (int64_t base = first; base < end; base += step, row += step, at += stride) {
            now = next;
            ask(row + step, at + stride);
            work(row, at, row < end);
        }
    }
    if constexpr (MODE == kRmsBwd) op.give_gradient(a, reinterpret_cast<float*>(smem));
}

// ---------------------------------------------------------------------------------------- host

struct RmsPlan {
    bool warp, odd;
    int v, k, team, threads;
};
// Vectors of 16 bytes where every row begins on one, else of 4 bytes (two 16-bit values; of an odd number all but one) or single values.  Teams as small as their
// threads' 16 values allow, so that a warp has several narrow rows at work, but so many threads that there is work for every SM.
inline RmsPlan rms_plan(int64_t rows, int width, int size, uintptr_t any, int sms) {
    RmsPlan p;
    const uintptr_t row = uintptr_t(width) * size | any;
    p.odd = size == 2 && width % 2 == 1 && width > 1 && any % 4 == 0;
    p.v = row % 16 == 0 ? 16 / size : p.odd || row % 4 == 0 ? 4 / size : 1;
    const int vecs = p.odd ? width / 2 : (width + p.v - 1) / p.v, most = kValues / p.v;
    p.warp = vecs <= 32 * most;
    p.k = most;
    if (p.warp) {
        p.team = std::max(1, 32 / (p.v * size));  // 32 bytes together
        while (p.team * most < vecs || (p.team < 32 && p.team < vecs && rows * p.team < int64_t(sms) * 1024)) p.team *= 2;
        while (p.k > 1 && p.team * (p.k / 2) >= vecs) p.k /= 2;
        if (p.k == 16 && p.team * 12 >= vecs) p.k = 12;
        p.threads = 256;
    } else {
        if (p.v == 1) p.k = 8;  // single values take a register each
        p.threads = p.team = ((vecs + p.k - 1) / p.k + 31) / 32 * 32;
    }
    return p;
}

// f(V, K, WARP) with the plan's values as types.
template <typename T, typename F>
cudaError_t by_plan(const RmsPlan& p, F f) {
#define UVU_AT(V_, K_, W_) \
    if (p.v == V_ && p.k == K_ && p.warp == W_) \
        return f(std::integral_constant<int, V_>(), std::integral_constant<int, K_>(), std::integral_constant<bool, W_>());
    if constexpr (sizeof(T) == 4) {
        UVU_AT(4, 1, true) UVU_AT(4, 2, true) UVU_AT(4, 4, true) UVU_AT(4, 4, false)
    } else {
        UVU_AT(8, 1, true) UVU_AT(8, 2, true) UVU_AT(8, 2, false)
        UVU_AT(2, 1, true) UVU_AT(2, 2, true) UVU_AT(2, 4, true) UVU_AT(2, 8, true) UVU_AT(2, 8, false)
    }
    UVU_AT(1, 1, true) UVU_AT(1, 2, true) UVU_AT(1, 4, true) UVU_AT(1, 8, true) UVU_AT(1, 12, true) UVU_AT(1, 16, true) UVU_AT(1, 8, false)
#undef UVU_AT
    return cudaErrorInvalidValue;
}

// Most blocks of the gradient, whose sums the workspace holds: so many on an SM, or more where a team's sums would get long.
inline int bwd_resident_most(const RmsPlan& p) { return std::max(8, 1024 / p.threads); }
inline int64_t bwd_blocks_most(const RmsPlan& p, int64_t rows, int sms) {
    const int64_t teams = p.threads / p.team;
    return std::min((rows + teams - 1) / teams, 1 + std::max(int64_t(sms) * bwd_resident_most(p), (rows + kTeamRows * teams - 1) / (kTeamRows * teams)));
}

template <typename T, RmsMode MODE>
cudaError_t rms_launch(RmsArgs a, int sms, cudaStream_t st, int64_t* partials) {
    constexpr bool kQuant = MODE == kRmsQuant || MODE == kRmsQuantAny;
    uintptr_t any = 0;
    for (const void* t : {a.in[0], a.in[1], a.in[2], static_cast<const void*>(a.out[0]), static_cast<const void*>(a.out[1])})
        any |= reinterpret_cast<uintptr_t>(t) * (kQuant && t == a.out[0] ? sizeof(T) : 1);
    const RmsPlan p = rms_plan(a.rows, a.width, sizeof(T), any, sms);
    if constexpr (MODE == kRmsQuant) {
        const int lanes = a.group / p.v;
        const bool even = !p.odd && a.group % p.v == 0 && (a.group & (a.group - 1)) == 0;
        if (a.group < a.width && !(even && (lanes <= std::min(p.team, 32) || (p.warp && p.team == 32))))
            return rms_launch<T, kRmsQuantAny>(a, sms, st, partials);
    }
    a.team = p.team;
    a.n_in = MODE == kRmsBwd ? (a.in[2] ? 3 : 2) : a.in[1] ? 2 : 1;
    a.slot = p.v * int(sizeof(T)) == 16 ? a.width * int(sizeof(T)) : 0;  // rows off 16 bytes have no places
    const int64_t teams = p.threads / p.team;
    const size_t one = size_t(teams) * a.n_in * a.slot;  // a row for each team
    return by_plan<T>(p, [&](auto v, auto k, auto warp) {
        constexpr int V = decltype(v)::value, K = decltype(k)::value;
        constexpr bool W = decltype(warp)::value;
        auto kernel = rms_kernel<T, V, K, W, kCut, MODE>;
        const bool full = V * sizeof(T) == 16 && p.team * p.k * p.v == a.width;
        if constexpr (V * sizeof(T) == 16)
            if (full) kernel = rms_kernel<T, V, K, W, kFull, MODE>;
        if constexpr (V == 2 && sizeof(T) == 2)
            if (p.odd) kernel = rms_kernel<T, V, K, W, kOdd, MODE>;
        static std::atomic<int> known[2];  // registers of a thread, of the other end than kCut too: the same on every device
        int regs = known[full || p.odd].load(std::memory_order_relaxed);
        if (regs == 0) {
            cudaFuncAttributes f;
            cudaError_t e = cudaFuncGetAttributes(&f, kernel);
            if (e != cudaSuccess) return e;
            known[full || p.odd].store(regs = std::max(1, f.numRegs), std::memory_order_relaxed);
        }
        auto smem_of = [&](int ahead) {
            const size_t b = one * (ahead + 1) + (MODE == kRmsQuantAny ? size_t(teams) * a.groups * 8 : 0);
            return MODE == kRmsBwd ? std::max(b, size_t(teams) * a.width * 4) : b;
        };
        auto resident = [&](size_t smem) {
            return std::max(1, std::min({MODE == kRmsBwd ? bwd_resident_most(p) : 32, 2048 / p.threads, 65536 / ((regs + 7) / 8 * 8 * p.threads), int((227 << 10) / (smem + 1280))}));
        };
        // three rows ahead where every team has several, else so many blocks as there is work for
        a.ahead = smem_of(kAhead) <= kRowsSmem && a.rows >= sms * resident(smem_of(kAhead)) * teams * (kAhead + 1) ? kAhead : 1;
        const size_t smem = smem_of(a.ahead);
        if (smem > 40 << 10) {  // with what is static, 48 KB need no leave
            cudaError_t e = allow_most_smem(kernel, smem);
            if (e != cudaSuccess) return e;
        }
        int64_t blocks = std::min<int64_t>((a.rows + teams - 1) / teams, int64_t(sms) * resident(smem));
        if (MODE == kRmsBwd) blocks = std::max(blocks, (a.rows + kTeamRows * teams - 1) / (kTeamRows * teams));
        if (p.odd && !p.warp) {
            if (blocks < a.rows) blocks += blocks & 1;  // a block's rows are so many apart
        } else if (MODE == kRmsBwd) {
            a.block_rows = ((a.rows + blocks - 1) / blocks + teams - 1) / teams * teams;
            blocks = (a.rows + a.block_rows - 1) / a.block_rows;
        }
        if (partials) *partials = blocks;
        kernel<<<unsigned(blocks), p.threads, smem, st>>>(a);
        return cudaGetLastError();
    });
}

inline RmsArgs rms_args(const RmsShape& s) {
    RmsArgs a = {};
    a.rows = s.rows;
    a.width = s.channels * s.inner;
    a.inner = s.inner;
    a.eps = float(s.eps);
    return a;
}
inline RmsArgs rms_fwd_args(const RmsShape& s, const void* x, const void* residual, const float* gamma, void* h, void* y, float* rstd) {
    RmsArgs a = rms_args(s);
    a.in[0] = x, a.in[1] = residual, a.gamma = gamma, a.out[0] = y, a.out[1] = h, a.rstd = rstd;
    return a;
}
inline RmsArgs rms_quant_args(const RmsShape& s, int group, const void* x, const void* residual, const float* gamma, void* h, void* q,
                              float* scales) {
    RmsArgs a = rms_args(s);
    a.in[0] = x, a.in[1] = residual, a.gamma = gamma, a.out[0] = q, a.out[1] = h, a.scales = scales;
    a.group = group ? std::min(group, a.width) : a.width;
    a.groups = (a.width + a.group - 1) / a.group;
    return a;
}
inline RmsArgs rms_bwd_args(const RmsShape& s, const void* dy, const void* h, const float* gamma, const float* rstd, const void* dh, void* dx,
                            float* partial) {
    RmsArgs a = rms_args(s);
    a.in[0] = h, a.in[1] = dy, a.in[2] = dh, a.out[0] = dx, a.gamma = gamma;
    a.rstd = const_cast<float*>(rstd), a.partial = partial;
    return a;
}

}  // namespace
}  // namespace uvu
