// RMS norm with the residual's addition and an output of 8 bits with scales: see rms.h.
#include "rms.h"

namespace uvu {

cudaError_t launch_rms_quant(const RmsShape& s, int group, const void* x, const void* residual, const float* gamma, void* h, void* q,
                             float* scales, int sms, cudaStream_t st) {
    if (rms_wide(s)) return launch_rms_wide_quant(s, group, x, residual, gamma, h, q, scales, sms, st);
    const RmsArgs a = rms_quant_args(s, group, x, residual, gamma, h, q, scales);
    switch (s.dtype) {
        case UVU_F32: return rms_launch<float, kRmsQuant>(a, sms, st, nullptr);
        case UVU_BF16: return rms_launch<__nv_bfloat16, kRmsQuant>(a, sms, st, nullptr);
        case UVU_F16: return rms_launch<__half, kRmsQuant>(a, sms, st, nullptr);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace uvu
