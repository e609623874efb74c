// Host-side declarations of the tcgen05 GEMM on 8-bit codes (gemm_codes_tc.cu).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace ql {
namespace tc {

struct CodesGemm {
  const int8_t* x;  // [M, ldx]
  int64_t M, K, ldx;
  const int8_t* w;  // [N, ldw]
  int64_t N, ldw;
  const float* x_scale;
  const float* w_scale;
  int w_scale_len;
  const uint16_t* bias;  // nullable
  void* y;
  int64_t ldy;
  int out_type;       // QL_OUT_*
  uint8_t* scratch;   // codes_gemm_bytes: parts' sums, the tokens in f16
  unsigned* tickets;  // zero between calls
  uint32_t* status;
  uint32_t wait_limit;
};
size_t codes_gemm_bytes(int64_t M, int64_t N, int64_t K);
cudaError_t launch_codes_gemm(const CodesGemm& g, cudaStream_t st);

}  // namespace tc
}  // namespace ql
