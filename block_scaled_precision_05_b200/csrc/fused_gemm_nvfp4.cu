// fused_gemm_nvfp4.cu -- the NVFP4 entry of fused_gemm.cuh (one source per format: the kernels compile side by side).
#include "fused_gemm.cuh"

extern "C" int nvfp4_gemm_fused(const bsp_fused_gemm_desc* desc, bsp_stream_t stream) {
  return bsp::run_fused<bsp::kNVF4>(desc, stream);
}
