// RMS norm with the residual's addition: see rms.h.
#include "rms.h"

namespace uvu {

cudaError_t launch_rms_fwd(const RmsShape& s, const void* x, const void* residual, const float* gamma, void* h, void* y, float* rstd,
                           int sms, cudaStream_t st) {
    RmsArgs a = rms_args(s);
    a.in[0] = x, a.in[1] = residual, a.gamma = gamma, a.out[0] = y, a.out[1] = h, a.rstd = rstd;
    switch (s.dtype) {
        case UVU_F32: return rms_launch<float, kRmsFwd>(a, sms, st, nullptr);
        case UVU_BF16: return rms_launch<__nv_bfloat16, kRmsFwd>(a, sms, st, nullptr);
        case UVU_F16: return rms_launch<__half, kRmsFwd>(a, sms, st, nullptr);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace uvu
