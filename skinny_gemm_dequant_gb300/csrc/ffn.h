// Host-side declarations of the 4-bit group-scaled linear and the gated feed-forward block.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace ql {

// ------------------------------------------------------------------ skinny calls (kernels_ffn_skinny.cu)
struct FfnSkinnyArgs {
  const uint16_t* x;  // bf16 [M, ldx]
  int64_t ldx;
  int M, K;
  const uint8_t* w;  // packed 4-bit codes or bf16, [rows, ldw_bytes]
  int64_t ldw_bytes;
  int N;  // outputs: weight rows of a plain linear, columns I of a gated block (its rows are 2I)
  const uint16_t* scale;  // bf16 or fp16 bits [rows, lds] (4-bit weights only)
  int64_t lds;
  int scale_fp16;
  const uint8_t* zero;  // [rows, ldz] or null: 8
  int64_t ldz;
  int group_shift;        // log2 of the group size
  const uint16_t* bias;   // bf16 [N] or null (plain linear only)
  uint16_t* y;            // bf16 [M, ldy]
  int64_t ldy;
  float alpha, limit;     // activation of a gated block
};
// A forward without a checkpoint goes to the few-token kernel up to 16 tokens (17408 x 5120: 60 us,
// tcgen05 64), and with more while its CTAs (32 tokens, 16 outputs) are few: four per SM for one pass
// over the weights (32 x 8192 x 2048 18.0 us, tcgen05 17.8; 32 x 17408 x 5120 73 and 64), two for more
// (64 x 2056 x 4096 14.3 and 17.5; 64 x 520 x 1024 3.9 and 7.2; 40 x 4096 x 2048 16.7 and 13.0)
inline bool ffn_few_tokens(int64_t M, int64_t I) {
  return M <= 16 || (M + 31) / 32 * ((I + 15) / 16) <= (M <= 32 ? 4 : 2) * kNumSMs;
}
cudaError_t launch_ffn_skinny(const FfnSkinnyArgs& a, cudaStream_t st);
cudaError_t launch_int4(bool gated, const FfnSkinnyArgs& a, cudaStream_t st);  // kernels_int4.cu

// ------------------------------------------------------------------ tcgen05 path (ffn_tc.cu)
namespace tc {
struct FfnForward {
  const uint16_t* x;    // bf16 [M, ldx]
  const uint16_t* w13;  // bf16 [2I, ldw]
  int64_t M, H, I, ldx, ldw;
  uint16_t* h;  // bf16 [M, ldh]
  int64_t ldh;
  float alpha, limit;
  int save;           // QL_SAVE_*
  void* ckpt;         // [M, 2, I padded to 128] bf16 or int8
  float* ckpt_scale;  // [M, 2, I padded / 128] (int8)
  float* slots;       // workspace: ffn_forward_slots bytes
  unsigned* tickets;  // workspace: zero between calls
  uint32_t* status;
  uint32_t wait_limit;
};
size_t ffn_forward_slots(int64_t M, int64_t H, int64_t I);
size_t ffn_backward_slots(int64_t M, int64_t H, int64_t I);
cudaError_t launch_ffn_forward(const FfnForward& f, cudaStream_t st);

struct FfnBackward {
  const uint16_t* dh;  // bf16 [M, ld_dh]
  const uint16_t* x;
  const uint16_t* w13;
  int64_t M, H, I, ld_dh, ldx, ldw;
  int save;
  const void* ckpt;
  const float* ckpt_scale;
  float alpha, limit;
  uint16_t* dgu;   // workspace: bf16 [M, 2I]
  uint16_t* dx;    // bf16 [M, ld_dx] or null
  int64_t ld_dx;
  uint16_t* dw13;  // bf16 [2I, ld_dw] or null
  int64_t ld_dw;
  float* slots;  // workspace: ffn_backward_slots bytes
  unsigned* tickets;
  uint32_t* status;
  uint32_t wait_limit;
};
cudaError_t launch_ffn_backward(const FfnBackward& b, cudaStream_t st);

// ql_gated_ffn_plan's answer for gemm (QL_FFN_GEMM_*), mode as there
void ffn_plan(int gemm, int64_t M, int64_t H, int64_t I, int mode, int32_t* out);
}  // namespace tc

}  // namespace ql
