// The MXFP4 product of fp4 tokens, and the choice of the tokens' type (moe_mx_gemm.h; fp8 tokens have sources of
// their own, which are compiled beside these).
#include "moe_mx_gemm.h"

namespace moe {

hipError_t launch_gemm_mx(const GemmMxArgs& a, hipStream_t s) {
  if (a.a_dt == MOE_DT_FP4_E2M1) return run<DT_FP4>(a, s);
  return a.out_dt == MOE_DT_F32 ? launch_gemm_mx_wide(a, s) : launch_gemm_mx_fp8(a, s);
}

}  // namespace moe
