// C ABI of the 4-bit group-scaled linear and the gated feed-forward block (declared in
// include/qlinear.h): argument validation and dispatch.
#include <cmath>
#include <cstdio>

#include "../../include/qlinear.h"
#include "ffn.h"
#include "internal.h"

using namespace ql;

namespace {

constexpr size_t kTicketOff = 256;  // the zero region of every workspace

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
inline bool al2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1) == 0; }
inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

ql_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return QL_OK;
  fprintf(stderr, "qlinear: CUDA error %s\n", cudaGetErrorString(e));
  return QL_ERR_CUDA;
}

bool act_ok(float alpha, float limit) { return std::isfinite(alpha) && !std::isnan(limit) && limit >= 0.f; }

// the 4-bit linear's and the 4-bit gated block's common checks; rows = weight rows, n = outputs
ql_status int4_check(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint8_t* w, int64_t rows, int64_t n,
                     int64_t ldw_bytes, const uint16_t* scale, int scale_fmt, int64_t lds, const uint8_t* zero,
                     int64_t ldz, int64_t group, const uint16_t* y, int64_t ldy) {
  if (!x || !w || !scale || !y) return QL_ERR_INVALID_ARG;
  if (M < 1 || rows < 1 || K < 1 || ldx < K || ldw_bytes < cdiv(K, 2) || ldy < n || group < 1)
    return QL_ERR_INVALID_ARG;
  if (scale_fmt != QL_SCALE_BF16 && scale_fmt != QL_SCALE_FP16) return QL_ERR_INVALID_ARG;
  if (lds < cdiv(K, group) || (zero && ldz < cdiv(K, group))) return QL_ERR_INVALID_ARG;
  if (M > 65535 || rows > (1 << 30) || K > (1 << 28)) return QL_ERR_UNSUPPORTED;
  if (K % 32 != 0 || group < 32 || (group & (group - 1)) != 0 || group > (1 << 28)) return QL_ERR_UNSUPPORTED;
  if (!al16(x) || !al16(w) || !al2(scale) || !al2(y) || ldx % 8 != 0 || ldw_bytes % 16 != 0) return QL_ERR_ALIGNMENT;
  return QL_OK;
}

FfnSkinnyArgs int4_args(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint8_t* w, int64_t ldw_bytes,
                        const uint16_t* scale, int scale_fmt, int64_t lds, const uint8_t* zero, int64_t ldz,
                        int64_t group, uint16_t* y, int64_t ldy) {
  FfnSkinnyArgs a = {};
  a.x = x;
  a.ldx = ldx;
  a.M = (int)M;
  a.K = (int)K;
  a.w = w;
  a.ldw_bytes = ldw_bytes;
  a.scale = scale;
  a.lds = lds;
  a.scale_fp16 = scale_fmt == QL_SCALE_FP16;
  a.zero = zero;
  a.ldz = ldz;
  while ((int64_t(1) << a.group_shift) < group) ++a.group_shift;
  a.y = y;
  a.ldy = ldy;
  return a;
}

// the gated block's shapes, strides and alignments shared by both directions
ql_status ffn_check(int64_t M, int64_t H, int64_t I, int64_t ldx, int64_t ldw, float alpha, float limit) {
  if (M < 1 || H < 1 || I < 1 || ldx < H || ldw < H) return QL_ERR_INVALID_ARG;
  if (!act_ok(alpha, limit)) return QL_ERR_INVALID_ARG;
  if (M > (1 << 22) || H > (1 << 20) || I > (1 << 20) || H % 8 != 0 || I % 8 != 0) return QL_ERR_UNSUPPORTED;
  if (ldx % 8 != 0 || ldw % 8 != 0) return QL_ERR_ALIGNMENT;
  return QL_OK;
}

}  // namespace

extern "C" {

ql_status qlinear_int4(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint8_t* w, int64_t N,
                       int64_t ldw_bytes, const uint16_t* w_scale, int scale_fmt, int64_t lds, const uint8_t* w_zero,
                       int64_t ldz, int64_t group, const uint16_t* bias, uint16_t* y, int64_t ldy, ql_stream_t stream,
                       int* path_out) {
  if (path_out) *path_out = QL_PATH_NONE;
  const ql_status s = int4_check(x, M, K, ldx, w, N, N, ldw_bytes, w_scale, scale_fmt, lds, w_zero, ldz, group, y, ldy);
  if (s != QL_OK) return s;
  if (!al2(bias)) return QL_ERR_ALIGNMENT;
  FfnSkinnyArgs a = int4_args(x, M, K, ldx, w, ldw_bytes, w_scale, scale_fmt, lds, w_zero, ldz, group, y, ldy);
  a.N = (int)N;
  a.bias = bias;
  const cudaError_t e = launch_int4(false, a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_status(e);
  if (path_out) *path_out = QL_PATH_INT4_SKINNY;
  return QL_OK;
}

ql_status gated_ffn_int4(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint8_t* w13, int64_t I,
                         int64_t ldw_bytes, const uint16_t* w_scale, int scale_fmt, int64_t lds,
                         const uint8_t* w_zero, int64_t ldz, int64_t group, float swiglu_alpha, float swiglu_limit,
                         uint16_t* h, int64_t ldh, ql_stream_t stream, int* path_out) {
  if (path_out) *path_out = QL_PATH_NONE;
  if (!act_ok(swiglu_alpha, swiglu_limit)) return QL_ERR_INVALID_ARG;
  if (I > (1 << 29)) return QL_ERR_UNSUPPORTED;
  const ql_status s =
      int4_check(x, M, H, ldx, w13, 2 * I, I, ldw_bytes, w_scale, scale_fmt, lds, w_zero, ldz, group, h, ldh);
  if (s != QL_OK) return s;
  FfnSkinnyArgs a = int4_args(x, M, H, ldx, w13, ldw_bytes, w_scale, scale_fmt, lds, w_zero, ldz, group, h, ldh);
  a.N = (int)I;
  a.alpha = swiglu_alpha;
  a.limit = swiglu_limit;
  const cudaError_t e = launch_int4(true, a, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_status(e);
  if (path_out) *path_out = QL_PATH_GATED_FFN_INT4;
  return QL_OK;
}

ql_status gated_ffn(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint16_t* w13, int64_t I, int64_t ldw,
                    float swiglu_alpha, float swiglu_limit, uint16_t* h, int64_t ldh, int save, void* ckpt,
                    float* ckpt_scale, void* workspace, size_t workspace_bytes, ql_stream_t stream, int* path_out) {
  if (path_out) *path_out = QL_PATH_NONE;
  if (!x || !w13 || !h || ldh < I) return QL_ERR_INVALID_ARG;
  if (save != QL_SAVE_NONE && save != QL_SAVE_BF16 && save != QL_SAVE_INT8) return QL_ERR_INVALID_ARG;
  if (save != QL_SAVE_NONE && !ckpt) return QL_ERR_INVALID_ARG;
  if (save == QL_SAVE_INT8 && !ckpt_scale) return QL_ERR_INVALID_ARG;
  const ql_status s = ffn_check(M, H, I, ldx, ldw, swiglu_alpha, swiglu_limit);
  if (s != QL_OK) return s;
  if (!al16(x) || !al16(w13) || !al16(h) || !al16(ckpt) || !al4(ckpt_scale) || ldh % 8 != 0) return QL_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < ql_workspace_bytes(QL_OP_GATED_FFN, M, I, H, 0, 0)) return QL_ERR_WORKSPACE;
  if (!al16(workspace)) return QL_ERR_ALIGNMENT;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  const bool few = save == QL_SAVE_NONE && ffn_few_tokens(M, I);
  if (few) {
    FfnSkinnyArgs a = {};
    a.x = x;
    a.ldx = ldx;
    a.M = (int)M;
    a.K = (int)H;
    a.w = reinterpret_cast<const uint8_t*>(w13);
    a.ldw_bytes = ldw * 2;
    a.N = (int)I;
    a.y = h;
    a.ldy = ldh;
    a.alpha = swiglu_alpha;
    a.limit = swiglu_limit;
    e = launch_ffn_skinny(a, st);
  } else {
    tc::FfnForward f = {};
    f.x = x;
    f.w13 = w13;
    f.M = M;
    f.H = H;
    f.I = I;
    f.ldx = ldx;
    f.ldw = ldw;
    f.h = h;
    f.ldh = ldh;
    f.alpha = swiglu_alpha;
    f.limit = swiglu_limit;
    f.save = save;
    f.ckpt = ckpt;
    f.ckpt_scale = ckpt_scale;
    f.slots = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + workspace_zero_bytes());
    f.tickets = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(workspace) + kTicketOff);
    f.status = static_cast<uint32_t*>(workspace);
    f.wait_limit = wait_limit();
    e = tc::launch_ffn_forward(f, st);
  }
  if (e != cudaSuccess) return cuda_status(e);
  if (path_out) *path_out = few ? QL_PATH_GATED_FFN_SKINNY : QL_PATH_GATED_FFN_TCGEN05;
  return QL_OK;
}

ql_status gated_ffn_backward(const uint16_t* dh, int64_t ld_dh, const uint16_t* x, int64_t M, int64_t H, int64_t ldx,
                             const uint16_t* w13, int64_t I, int64_t ldw, float swiglu_alpha, float swiglu_limit,
                             int save, const void* ckpt, const float* ckpt_scale, uint16_t* dx, int64_t ld_dx,
                             uint16_t* dw13, int64_t ld_dw, void* workspace, size_t workspace_bytes,
                             ql_stream_t stream, int* path_out) {
  if (path_out) *path_out = QL_PATH_NONE;
  if (!dh || !ckpt || (!dx && !dw13) || (dx && !w13) || (dw13 && !x)) return QL_ERR_INVALID_ARG;
  if (save != QL_SAVE_BF16 && save != QL_SAVE_INT8) return QL_ERR_INVALID_ARG;
  if (save == QL_SAVE_INT8 && !ckpt_scale) return QL_ERR_INVALID_ARG;
  if (ld_dh < I || (dx && ld_dx < H) || (dw13 && ld_dw < H)) return QL_ERR_INVALID_ARG;
  const ql_status s = ffn_check(M, H, I, dw13 ? ldx : (H + 7) / 8 * 8, dx ? ldw : (H + 7) / 8 * 8, swiglu_alpha,
                                swiglu_limit);
  if (s != QL_OK) return s;
  if (!al16(dh) || !al16(ckpt) || !al4(ckpt_scale) || ld_dh % 8 != 0) return QL_ERR_ALIGNMENT;
  if (dx && (!al16(w13) || !al16(dx) || ld_dx % 8 != 0)) return QL_ERR_ALIGNMENT;
  if (dw13 && (!al16(x) || !al16(dw13) || ld_dw % 8 != 0)) return QL_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < ql_workspace_bytes(QL_OP_GATED_FFN_BWD, M, I, H, 0, 0)) return QL_ERR_WORKSPACE;
  if (!al16(workspace)) return QL_ERR_ALIGNMENT;
  tc::FfnBackward b = {};
  b.dh = dh;
  b.x = x;
  b.w13 = w13;
  b.M = M;
  b.H = H;
  b.I = I;
  b.ld_dh = ld_dh;
  b.ldx = ldx;
  b.ldw = ldw;
  b.save = save;
  b.ckpt = ckpt;
  b.ckpt_scale = ckpt_scale;
  b.alpha = swiglu_alpha;
  b.limit = swiglu_limit;
  uint8_t* regions = static_cast<uint8_t*>(workspace) + workspace_zero_bytes();
  b.dgu = reinterpret_cast<uint16_t*>(regions);
  b.slots = reinterpret_cast<float*>(regions + ((size_t)M * 2 * I * 2 + 255) / 256 * 256);
  b.tickets = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(workspace) + kTicketOff);
  b.dx = dx;
  b.ld_dx = ld_dx;
  b.dw13 = dw13;
  b.ld_dw = ld_dw;
  b.status = static_cast<uint32_t*>(workspace);
  b.wait_limit = wait_limit();
  const cudaError_t e = tc::launch_ffn_backward(b, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_status(e);
  if (path_out) *path_out = QL_PATH_GATED_FFN_BACKWARD;
  return QL_OK;
}

ql_status ql_gated_ffn_plan(int gemm, int64_t M, int64_t I, int64_t H, int mode, int32_t* out) {
  if (!out || gemm < QL_FFN_GEMM_FORWARD || gemm > QL_FFN_GEMM_DW) return QL_ERR_INVALID_ARG;
  if (gemm == QL_FFN_GEMM_FORWARD ? mode < QL_SAVE_NONE || mode > QL_SAVE_INT8 : mode != 0 && mode != 1)
    return QL_ERR_INVALID_ARG;
  const ql_status s = ffn_check(M, H, I, (H + 7) / 8 * 8, (H + 7) / 8 * 8, 1.f, 1.f);
  if (s != QL_OK) return s;
  for (int i = 0; i < 6; ++i) out[i] = 0;
  if (gemm == QL_FFN_GEMM_FORWARD && mode == QL_SAVE_NONE && ffn_few_tokens(M, I)) {
    out[5] = 1;
    return QL_OK;
  }
  tc::ffn_plan(gemm, M, H, I, mode, out);
  return QL_OK;
}

}  // extern "C"
