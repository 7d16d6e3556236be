// fused_gemm_nvfp4.cu -- the NVFP4 entry of fused_gemm.cuh (one source per format: the kernels compile side by side).
#include "fused_gemm.cuh"

extern "C" int nvfp4_gemm_fused(const bsp_fused_gemm_desc* desc, bsp_stream_t stream) {
  return bsp::run_fused<bsp::kNVF4>(desc, stream);
}

extern "C" int bsp_debug_fused_plan(int mxfp8, int grouped, int64_t E, int64_t M, int64_t N, int64_t K, int sm_count,
                                    int32_t* plan) {
  if (plan == nullptr || sm_count < 1 || E < 1 || M < 1 || N < 1 || K < 32 || K % 32 != 0) return BSP_ERR_INVALID_ARG;
  const bsp::FusedPlan p = bsp::plan_fused(sm_count, grouped != 0, E, M, N, bsp::ceil_div(mxfp8 ? K : K / 2, 128));
  plan[0] = p.ctas, plan[1] = p.tn, plan[2] = p.split;
  return BSP_OK;
}
