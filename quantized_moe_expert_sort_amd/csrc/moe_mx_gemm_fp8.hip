// The MXFP4 product of fp8 tokens, bf16 results (moe_mx_gemm.h).
#include "moe_mx_gemm.h"

namespace moe {

hipError_t launch_gemm_mx_fp8(const GemmMxArgs& a, hipStream_t s) { return run<DT_FP8>(a, s); }

}  // namespace moe
