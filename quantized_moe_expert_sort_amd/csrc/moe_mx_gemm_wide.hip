// The MXFP4 product of fp8 tokens, fp32 results (moe_mx_gemm.h).
#include "moe_mx_gemm.h"

namespace moe {

hipError_t launch_gemm_mx_wide(const GemmMxArgs& a, hipStream_t s) { return run<FP8_WIDE>(a, s); }

}  // namespace moe
