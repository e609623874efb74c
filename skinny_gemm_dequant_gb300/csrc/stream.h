// Host-side declarations of the weight-streaming kernels for few tokens (kernels_stream.cu,
// kernels_moe_few.cu): the mixture-of-experts layers on bf16, 8-bit and 4-bit weights and the linear on
// 8-bit codes.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace ql {

enum { STREAM_BF16 = 0, STREAM_INT8 = 1, STREAM_INT4 = 2 };
enum { STREAM_GATE_UP = 0, STREAM_LINEAR = 1 };

constexpr int kStreamRows = 64;       // weight rows of a tile
constexpr int kMoeMaxTokens = 64;     // of a mixture-of-experts call
constexpr int kMoeMaxTopk = 16;
constexpr int kMoeHandedBytes = 16640;
constexpr int kLinearTokens = 16;     // of a pass of LINEAR over the weights

// LINEAR's launch or, for more tokens and larger matrices, the GEMM's (gemm_codes.h).  LINEAR takes 5 us and a
// time that grows with passes, rows and (K + 3300); the GEMM hardly grows with few tokens.  Both sides in
// us: 17408x5120, 16 tokens 28 and 32, 32 tokens 42 and 33; 5120x5120, 32 tokens 20 and 22, 64 tokens 29
// and 25; 2048x4096, 64 tokens 16 and 21, 128 tokens 22 and 25, 192 tokens 30 and 24; 5120x512, 32 tokens
// 9 and 11, 64 tokens 14 and 12; 512x1024, 256 tokens 5 and 15.
inline bool linear_streams(int64_t M, int64_t N, int64_t K) {
  if (M <= kLinearTokens) return true;
  const int64_t rows = (M + kLinearTokens - 1) / kLinearTokens * N;
  return M <= 1024 && rows * (K + 3300) <= 24500 * (K < 3100 ? K + 2100 : 5200);
}

struct StreamArgs {
  const uint8_t* x;  // activations: bf16 rows (tokens; DOWN: h by pair), LINEAR: 8-bit codes
  int64_t ldx;       // bytes
  int K;             // summed elements
  const uint8_t* w;
  int64_t ldw, w_estride;  // bytes
  int N;                   // outputs: GATE_UP: I (2I rows of W13), DOWN: H, LINEAR: N
  const void* scale;       // INT4: bf16 / fp16 bits [rows, lds]; INT8: fp32 [rows]
  int64_t lds, s_estride;  // elements
  int scale_fp16;
  const uint8_t* zero;     // INT4: [rows, ldz] or null: 8
  int64_t ldz, z_estride;
  int group_shift;
  // routing (GATE_UP, DOWN)
  const uint16_t* logits;  // bf16 [M, E] or null
  const int32_t* ids;      // [M, topk] and fp32 weights, where logits are null
  const float* wts;
  int M, E, topk, renorm;
  int32_t* ids_out;  // nullable
  float* wts_out;
  float alpha, limit;
  uint16_t* h;  // GATE_UP writes bf16 [M topk, ldh]
  int64_t ldh;
  void* handed;       // kMoeHandedBytes that GATE_UP writes for DOWN (moe_dispatch.cuh)
  float* heads;       // DOWN: down_head_bytes
  unsigned* amax;     // INT8: [M topk] bits of max|h|, zero between calls
  unsigned* tickets;  // zero between calls
  float* slots;       // sums of tiles that CTAs share
  // DOWN, LINEAR
  void* y;
  int64_t ldy;
  int out_type;          // LINEAR: QL_OUT_*
  const uint16_t* bias;  // LINEAR
  const float* x_scale;  // LINEAR: [M]
};

// codes and scales of tokens (kernels_codes.cu)
cudaError_t launch_token_codes(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int8_t* codes, float* scale,
                               cudaStream_t st);
// kernels_stream.cu: GATE_UP of any call, LINEAR of what linear_streams says
cudaError_t launch_gate_up(int fmt, const StreamArgs& a, cudaStream_t st);
cudaError_t launch_linear(const StreamArgs& a, cudaStream_t st);
// kernels_moe_few.cu: GATE_UP while the tokens fit in shared memory, DOWN
bool gate_up_few_takes(int fmt, const StreamArgs& a);
cudaError_t launch_gate_up_few(int fmt, const StreamArgs& a, cudaStream_t st);
cudaError_t launch_down(int fmt, const StreamArgs& a, cudaStream_t st);
size_t down_head_bytes(int64_t M);
size_t stream_slot_bytes(int64_t M);
// of QL_OP_INT8_CODES and QL_OP_MOE_FEW (api_stream.cu)
size_t stream_workspace_bytes(int op, int64_t M, int64_t N, int64_t K, int E, int topk);

}  // namespace ql
