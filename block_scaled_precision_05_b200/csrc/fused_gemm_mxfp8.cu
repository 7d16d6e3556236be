// fused_gemm_mxfp8.cu -- the MXFP8 entry of fused_gemm.cuh (one source per format: the kernels compile side by side).
#include "fused_gemm.cuh"

extern "C" int mxfp8_gemm_fused(const bsp_fused_gemm_desc* desc, bsp_stream_t stream) {
  return bsp::run_fused<bsp::kMXF8>(desc, stream);
}
