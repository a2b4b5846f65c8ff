// The gradient of the RMS norm: see rms.h.
#include "rms.h"

namespace uvu {
namespace {

// d_gamma[c] = sum over the blocks of partial[b][c]: 32 channels a block, 32 threads for each.
__global__ void __launch_bounds__(1024) rms_join_kernel(const float* partial, int blocks, int channels, float* out) {
    __shared__ float s[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the sums are there
    const int c = blockIdx.x * 32 + threadIdx.x;
    float sum = 0.f;
    if (c < channels) {
        int b = threadIdx.y;
        for (; b + 96 < blocks; b += 128) {  // four loads on their way
            const float* p = partial + int64_t(b) * channels + c;
            const float v0 = p[0], v1 = p[int64_t(32) * channels], v2 = p[int64_t(64) * channels], v3 = p[int64_t(96) * channels];
            sum += (v0 + v1) + (v2 + v3);
        }
        for (; b < blocks; b += 32) sum += partial[int64_t(b) * channels + c];
    }
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    sum = s[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    const int out_c = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && out_c < channels) out[out_c] = sum;
}

}  // namespace

size_t rms_workspace(const RmsShape& s, int sms) {
    if (s.rows == 0) return 0;
    if (rms_wide(s)) return size_t(rms_wide_blocks(s.rows, sms)) * s.channels * 4;
    // the tensors' alignment is not known here: the most blocks of any
    int64_t most = 0;
    for (uintptr_t any : {0, 4, 2, 1})
        most = std::max(most, bwd_blocks_most(rms_plan(s.rows, s.channels * s.inner, s.dtype == UVU_F32 ? 4 : 2, any, sms), s.rows, sms));
    return size_t(most) * s.channels * 4;
}

cudaError_t launch_rms_bwd(const RmsShape& s, const void* dy, const void* h, const float* gamma, const float* rstd, const void* dh,
                           void* dx, float* dgamma, void* ws, int sms, cudaStream_t st) {
    if (s.rows == 0) return cudaMemsetAsync(dgamma, 0, size_t(s.channels) * 4, st);
    const RmsArgs a = rms_bwd_args(s, dy, h, gamma, rstd, dh, dx, static_cast<float*>(ws));
    int64_t blocks = 0;
    cudaError_t e = cudaErrorInvalidValue;
    if (rms_wide(s)) {
        e = launch_rms_wide_bwd(s, dy, h, gamma, rstd, dh, dx, a.partial, sms, st, &blocks);
    } else {
        switch (s.dtype) {
            case UVU_F32: e = rms_launch<float, kRmsBwd>(a, sms, st, &blocks); break;
            case UVU_BF16: e = rms_launch<__nv_bfloat16, kRmsBwd>(a, sms, st, &blocks); break;
            case UVU_F16: e = rms_launch<__half, kRmsBwd>(a, sms, st, &blocks); break;
            default: break;
        }
    }
    if (e != cudaSuccess) return e;
    // it may begin while the last blocks of the sums run, and waits for them
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((s.channels + 31) / 32);
    c.blockDim = dim3(32, 32);
    c.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, rms_join_kernel, static_cast<const float*>(a.partial), int(blocks), s.channels, dgamma);
}

}  // namespace uvu
