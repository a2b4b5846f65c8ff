// RMS norm with the residual's addition: see rms.h.
#include "rms.h"

namespace uvu {

cudaError_t launch_rms_fwd(const RmsShape& s, const void* x, const void* residual, const float* gamma, void* h, void* y, float* rstd,
                           int sms, cudaStream_t st) {
    if (rms_wide(s)) return launch_rms_wide_fwd(s, x, residual, gamma, h, y, rstd, sms, st);
    const RmsArgs a = rms_fwd_args(s, x, residual, gamma, h, y, rstd);
    switch (s.dtype) {
        case UVU_F32: return rms_launch<float, kRmsFwd>(a, sms, st, nullptr);
        case UVU_BF16: return rms_launch<__nv_bfloat16, kRmsFwd>(a, sms, st, nullptr);
        case UVU_F16: return rms_launch<__half, kRmsFwd>(a, sms, st, nullptr);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace uvu
