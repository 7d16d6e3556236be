// fused_gemm_nvfp4.cu -- the NVFP4 entries of fused_gemm.cuh (one source per format: the kernels compile side by side).
#include "fused_gemm.cuh"

extern "C" {

int nvfp4_gemm_fused(const uint8_t* A, const uint8_t* sfA, const uint8_t* B, const uint8_t* sfB, int64_t M, int64_t N,
                     int64_t K, const float* alpha, const float* row_scale, const uint16_t* bias, int activation,
                     int gated, const void* residual, int64_t ld_residual, void* D, int d_dtype, int64_t ld_d,
                     bsp_stream_t stream) {
  return bsp::run_fused<bsp::kNVF4>(A, sfA, B, sfB, nullptr, 1, M, N, K, alpha, row_scale, bias, activation, gated,
                                    residual, ld_residual, D, d_dtype, ld_d, stream);
}

int nvfp4_grouped_gemm(const uint8_t* A, const uint8_t* sfA, const uint8_t* B, const uint8_t* sfB,
                       const int32_t* offsets, int64_t E, int64_t M, int64_t N, int64_t K, const float* alpha,
                       const float* row_scale, const uint16_t* bias, int activation, int gated, void* D, int d_dtype,
                       int64_t ld_d, bsp_stream_t stream) {
  if (offsets == nullptr && M > 0 && N > 0) return BSP_ERR_INVALID_ARG;
  return bsp::run_fused<bsp::kNVF4>(A, sfA, B, sfB, offsets, E, M, N, K, alpha, row_scale, bias, activation, gated,
                                    nullptr, 0, D, d_dtype, ld_d, stream);
}

}  // extern "C"
