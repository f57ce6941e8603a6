// Instances of the products of ffn_gemm.h for one operand type: FFN_DTYPE is a
// conv_dtype_t (fp32 0, bf16 1, fp16 2, e4m3 3).
#include "ffn_gemm.h"

namespace convlower {

#if FFN_DTYPE == 3
hipError_t launch_ffn_gated_fp8(const FfnGemmArgs &a, int out_dtype, hipStream_t st) {
    return out_dtype == CONV_DTYPE_FP16 ? ffn_run<uint8_t, _Float16, FFN_SCALED, false, false>(a, st)
                                        : ffn_run<uint8_t, uint16_t, FFN_SCALED, false, false>(a, st);
}
#else
#if FFN_DTYPE == 0
#define FFN_NAME(x) x##_f32
typedef float ffn_t;
#elif FFN_DTYPE == 1
#define FFN_NAME(x) x##_bf16
typedef uint16_t ffn_t;
#else
#define FFN_NAME(x) x##_f16
typedef _Float16 ffn_t;
#endif
hipError_t FFN_NAME(launch_ffn_gated)(const FfnGemmArgs &a, bool saving, hipStream_t st) {
    return saving ? ffn_run<ffn_t, ffn_t, FFN_SAVING, false, false>(a, st)
                  : ffn_run<ffn_t, ffn_t, FFN_GATED, false, false>(a, st);
}
hipError_t FFN_NAME(launch_ffn_dx)(const FfnGemmArgs &a, hipStream_t st) {
    return ffn_run<ffn_t, ffn_t, FFN_PLAIN, false, true>(a, st);
}
hipError_t FFN_NAME(launch_ffn_dw)(const FfnGemmArgs &a, hipStream_t st) {
    return ffn_run<ffn_t, ffn_t, FFN_PLAIN, true, true>(a, st);
}
#endif

}  // namespace convlower
