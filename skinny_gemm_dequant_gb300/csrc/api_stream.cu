// C ABI of the 8-bit-code linear and of the mixture-of-experts layers for a few tokens (declared in
// include/qlinear.h): argument validation and dispatch.
#include <cmath>
#include <cstdio>

#include "../../include/qlinear.h"
#include "gemm_codes.h"
#include "internal.h"
#include "stream.h"

using namespace ql;

namespace {

constexpr size_t kTicketOff = 256;          // the zero region of every workspace: tickets,
constexpr size_t kAmaxOff = 256 + 4096;     // then the rows' maxima of moe_int8
static_assert((kNumSMs + 1) * 4 <= 4096 && kMoeMaxTokens * kMoeMaxTopk * 4 <= (1 << 20) - 4096, "zero region");

template <int N>
bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & (N - 1)) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t al256(size_t b) { return (b + 255) & ~size_t(255); }

ql_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return QL_OK;
  fprintf(stderr, "qlinear: CUDA error %s\n", cudaGetErrorString(e));
  return QL_ERR_CUDA;
}
template <class T>
T* at(void* workspace, size_t off) { return reinterpret_cast<T*>(static_cast<uint8_t*>(workspace) + off); }

// what the mixture-of-experts calls share
struct Moe {
  const uint16_t* x;
  int64_t M, H, ldx;
  const uint16_t* logits;
  const int32_t* ids;
  const float* wts;
  int E, topk, renorm;
  int64_t I;
  float alpha, limit;
  int32_t* ids_out;
  float* wts_out;
  uint16_t* h_out;
  uint16_t* y;
  int64_t ldy;
  void* ws;
  size_t ws_bytes;
};
struct Matrix {  // a projection's weights, rows x k
  const void* w;
  int64_t ldw, estride;  // bytes
};

// k_align: elements of 16 bytes of a weight row; esize2: twice the bytes of an element
ql_status moe_check(const Moe& a, const Matrix& w13, const Matrix& w2, int k_align, int esize2) {
  if (!a.x || !w13.w || !w2.w || !a.y) return QL_ERR_INVALID_ARG;
  if (!std::isfinite(a.alpha) || std::isnan(a.limit) || a.limit < 0.f) return QL_ERR_INVALID_ARG;
  if ((a.logits == nullptr) == (a.ids == nullptr) || (a.ids && !a.wts)) return QL_ERR_INVALID_ARG;
  if (a.M < 1 || a.H < 1 || a.I < 1 || a.E < 1 || a.topk < 1 || a.ldx < a.H || a.ldy < a.H) return QL_ERR_INVALID_ARG;
  if (a.M > kMoeMaxTokens || a.topk > kMoeMaxTopk || a.topk > a.E || a.E > 1024) return QL_ERR_UNSUPPORTED;
  if (a.H % k_align != 0 || a.I % k_align != 0 || a.H > 32768 || a.I > 32768) return QL_ERR_UNSUPPORTED;
  if (w13.ldw < a.H * esize2 / 2 || w2.ldw < a.I * esize2 / 2 || w13.estride < 0 || w2.estride < 0)
    return QL_ERR_INVALID_ARG;
  if (!aligned<16>(a.x) || !aligned<16>(w13.w) || !aligned<16>(w2.w) || a.ldx % 8 != 0 || w13.ldw % 16 != 0 ||
      w2.ldw % 16 != 0 || w13.estride % 16 != 0 || w2.estride % 16 != 0)
    return QL_ERR_ALIGNMENT;
  if (!aligned<2>(a.logits) || !aligned<4>(a.ids) || !aligned<4>(a.wts) || !aligned<4>(a.ids_out) ||
      !aligned<4>(a.wts_out) || !aligned<2>(a.h_out) || !aligned<2>(a.y))
    return QL_ERR_ALIGNMENT;
  if (!a.ws || a.ws_bytes < ql_workspace_bytes(QL_OP_MOE_FEW, a.M, a.H, a.I, a.E, a.topk)) return QL_ERR_WORKSPACE;
  if (!aligned<16>(a.ws)) return QL_ERR_ALIGNMENT;
  return QL_OK;
}

StreamArgs moe_args(const Moe& a) {
  StreamArgs s = {};
  s.logits = a.logits;
  s.ids = a.ids;
  s.wts = a.wts;
  s.M = (int)a.M;
  s.E = a.E;
  s.topk = a.topk;
  s.renorm = a.renorm;
  s.ids_out = a.ids_out;
  s.wts_out = a.wts_out;
  s.alpha = a.alpha;
  s.limit = a.limit;
  s.tickets = at<unsigned>(a.ws, kTicketOff);
  s.amax = at<unsigned>(a.ws, kAmaxOff);
  s.slots = at<float>(a.ws, workspace_zero_bytes());
  s.handed = at<uint8_t>(a.ws, workspace_zero_bytes() + al256(stream_slot_bytes(a.M)));
  s.heads = reinterpret_cast<float*>(static_cast<uint8_t*>(s.handed) + kMoeHandedBytes);
  s.h = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(s.heads) + al256(down_head_bytes(a.M)));
  s.ldh = cdiv(a.I, 8) * 8;
  return s;
}

void set_matrix(StreamArgs& s, const Matrix& w) {
  s.w = static_cast<const uint8_t*>(w.w);
  s.ldw = w.ldw;
  s.w_estride = w.estride;
}

// the two launches; gu and dn hold their weights' scales already
ql_status moe_run(int fmt, const Moe& a, const Matrix& w13, const Matrix& w2, StreamArgs& gu, StreamArgs& dn,
                  cudaStream_t st, int path, int* path_out) {
  set_matrix(gu, w13);
  gu.x = reinterpret_cast<const uint8_t*>(a.x);
  gu.ldx = a.ldx * 2;
  gu.K = (int)a.H;
  gu.N = (int)a.I;
  set_matrix(dn, w2);
  dn.x = reinterpret_cast<const uint8_t*>(dn.h);
  dn.ldx = dn.ldh * 2;
  dn.K = (int)a.I;
  dn.N = (int)a.H;
  dn.y = a.y;
  dn.ldy = a.ldy;
  cudaError_t e = cudaSuccess;
  if (a.h_out) {  // GATE_UP writes no row of a padding pair: the caller gets zeros there, not an earlier call's h
    e = cudaMemsetAsync(gu.h, 0, (size_t)a.M * a.topk * gu.ldh * 2, st);
    if (e != cudaSuccess) return cuda_status(e);
  }
  e = gate_up_few_takes(fmt, gu) ? launch_gate_up_few(fmt, gu, st) : launch_gate_up(fmt, gu, st);
  if (e != cudaSuccess) return cuda_status(e);
  e = launch_down(fmt, dn, st);
  if (e != cudaSuccess) {
    // the maxima that GATE_UP left are not taken back: what is zero between calls is made so
    cudaMemsetAsync(gu.amax, 0, (size_t)a.M * a.topk * 4, st);
    return cuda_status(e);
  }
  if (a.h_out) {
    e = cudaMemcpy2DAsync(a.h_out, a.I * 2, dn.h, dn.ldh * 2, a.I * 2, a.M * a.topk, cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) return cuda_status(e);
  }
  if (path_out) *path_out = path;
  return QL_OK;
}

}  // namespace

namespace ql {
size_t stream_workspace_bytes(int op, int64_t M, int64_t N, int64_t K, int E, int topk) {
  if (op == QL_OP_INT8_CODES) {
    if (M > (1 << 22) || N > (1 << 24) || K > 131056 || M < 1 || N < 1 || K < 1) return workspace_zero_bytes();  // refused
    return workspace_zero_bytes() + (linear_streams(M, N, K) ? stream_slot_bytes(1) : tc::codes_gemm_bytes(M, N, K));
  }
  if (E <= 0 || topk <= 0) return 0;
  if (M > kMoeMaxTokens || topk > kMoeMaxTopk || K > 32768) return workspace_zero_bytes();  // refused
  return workspace_zero_bytes() + al256(stream_slot_bytes(M)) +
         kMoeHandedBytes + al256(down_head_bytes(M)) + (size_t)M * topk * cdiv(K, 8) * 8 * 2;
}
}  // namespace ql

extern "C" {

ql_status quantize_int8(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int8_t* codes, float* scale,
                        ql_stream_t stream) {
  if (!x || !codes || !scale || M < 1 || K < 1 || ldx < K) return QL_ERR_INVALID_ARG;
  if (M > (1 << 22) || K > (1 << 20) || K % 8 != 0) return QL_ERR_UNSUPPORTED;
  if (!aligned<16>(x) || !aligned<16>(codes) || !aligned<4>(scale) || ldx % 8 != 0) return QL_ERR_ALIGNMENT;
  return cuda_status(launch_token_codes(x, M, K, ldx, codes, scale, (cudaStream_t)stream));
}

ql_status qlinear_int8(const int8_t* x_q, int64_t M, int64_t K, int64_t ldx, const float* x_scale, const int8_t* w,
                       int64_t N, int64_t ldw, const float* w_scale, int64_t w_scale_len, const uint16_t* bias,
                       int out_type, void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                       ql_stream_t stream, int* path_out) {
  if (path_out) *path_out = QL_PATH_NONE;
  if (!x_q || !x_scale || !w || !w_scale || !y) return QL_ERR_INVALID_ARG;
  if (M < 1 || N < 1 || K < 1 || ldx < K || ldw < K || ldy < N || (w_scale_len != 1 && w_scale_len != N))
    return QL_ERR_INVALID_ARG;
  if (out_type < QL_OUT_BF16 || out_type > QL_OUT_FP32) return QL_ERR_INVALID_ARG;
  if (M > (1 << 22) || N > (1 << 24) || K % 16 != 0 || K > 131056) return QL_ERR_UNSUPPORTED;
  if (!aligned<16>(x_q) || !aligned<16>(w) || ldx % 16 != 0 || ldw % 16 != 0 || !aligned<4>(x_scale) ||
      !aligned<4>(w_scale) || !aligned<2>(bias) || !(out_type == QL_OUT_FP32 ? aligned<4>(y) : aligned<2>(y)))
    return QL_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < ql_workspace_bytes(QL_OP_INT8_CODES, M, N, K, 0, 0)) return QL_ERR_WORKSPACE;
  if (!aligned<16>(workspace)) return QL_ERR_ALIGNMENT;
  if (!linear_streams(M, N, K)) {
    tc::CodesGemm g = {};
    g.x = x_q;
    g.M = M;
    g.K = K;
    g.ldx = ldx;
    g.w = w;
    g.N = N;
    g.ldw = ldw;
    g.x_scale = x_scale;
    g.w_scale = w_scale;
    g.w_scale_len = (int)w_scale_len;
    g.bias = bias;
    g.y = y;
    g.ldy = ldy;
    g.out_type = out_type;
    g.scratch = at<uint8_t>(workspace, workspace_zero_bytes());
    g.tickets = at<unsigned>(workspace, kTicketOff);
    g.status = at<uint32_t>(workspace, 0);
    g.wait_limit = wait_limit();
    const cudaError_t e = tc::launch_codes_gemm(g, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_status(e);
    if (path_out) *path_out = QL_PATH_INT8_CODES_TCGEN05;
    return QL_OK;
  }
  StreamArgs s = {};
  s.x = reinterpret_cast<const uint8_t*>(x_q);
  s.ldx = ldx;
  s.K = (int)K;
  s.M = (int)M;
  s.w = reinterpret_cast<const uint8_t*>(w);
  s.ldw = ldw;
  s.N = (int)N;
  s.scale = w_scale;
  s.lds = w_scale_len > 1;
  s.x_scale = x_scale;
  s.bias = bias;
  s.out_type = out_type;
  s.y = y;
  s.ldy = ldy;
  s.tickets = at<unsigned>(workspace, kTicketOff);
  s.slots = at<float>(workspace, workspace_zero_bytes());
  const cudaError_t e = launch_linear(s, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_status(e);
  if (path_out) *path_out = QL_PATH_INT8_CODES_SKINNY;
  return QL_OK;
}

ql_status moe_bf16(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint16_t* router_logits,
                   const int32_t* topk_ids_in, const float* topk_w_in, int E, int topk, int renormalize,
                   const uint16_t* w13, int64_t ldw13, int64_t w_estride13, const uint16_t* w2, int64_t ldw2,
                   int64_t w_estride2, int64_t I, float swiglu_alpha, float swiglu_limit, int32_t* topk_ids_out,
                   float* topk_w_out, uint16_t* h_out, uint16_t* y, int64_t ldy, void* workspace,
                   size_t workspace_bytes, ql_stream_t stream, int* path_out) {
  if (path_out) *path_out = QL_PATH_NONE;
  const Moe a = {x, M, H, ldx, router_logits, topk_ids_in, topk_w_in, E, topk, renormalize, I, swiglu_alpha,
                 swiglu_limit, topk_ids_out, topk_w_out, h_out, y, ldy, workspace, workspace_bytes};
  const Matrix a13 = {w13, ldw13 * 2, w_estride13 * 2}, a2 = {w2, ldw2 * 2, w_estride2 * 2};
  if (const ql_status s = moe_check(a, a13, a2, 8, 4); s != QL_OK) return s;
  StreamArgs gu = moe_args(a), dn = gu;
  return moe_run(STREAM_BF16, a, a13, a2, gu, dn, (cudaStream_t)stream, QL_PATH_MOE_BF16, path_out);
}

ql_status moe_int8(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint16_t* router_logits,
                   const int32_t* topk_ids_in, const float* topk_w_in, int E, int topk, int renormalize,
                   const int8_t* w13, int64_t ldw13, int64_t w_estride13, const float* s13, const int8_t* w2,
                   int64_t ldw2, int64_t w_estride2, const float* s2, int64_t I, float swiglu_alpha,
                   float swiglu_limit, int32_t* topk_ids_out, float* topk_w_out, uint16_t* h_out, uint16_t* y,
                   int64_t ldy, void* workspace, size_t workspace_bytes, ql_stream_t stream, int* path_out) {
  if (path_out) *path_out = QL_PATH_NONE;
  const Moe a = {x, M, H, ldx, router_logits, topk_ids_in, topk_w_in, E, topk, renormalize, I, swiglu_alpha,
                 swiglu_limit, topk_ids_out, topk_w_out, h_out, y, ldy, workspace, workspace_bytes};
  const Matrix a13 = {w13, ldw13, w_estride13}, a2 = {w2, ldw2, w_estride2};
  if (!s13 || !s2) return QL_ERR_INVALID_ARG;
  if (const ql_status s = moe_check(a, a13, a2, 16, 2); s != QL_OK) return s;
  if (!aligned<4>(s13) || !aligned<4>(s2)) return QL_ERR_ALIGNMENT;
  StreamArgs gu = moe_args(a), dn = gu;
  gu.scale = s13;
  gu.s_estride = 2 * I;
  dn.scale = s2;
  dn.s_estride = H;
  return moe_run(STREAM_INT8, a, a13, a2, gu, dn, (cudaStream_t)stream, QL_PATH_MOE_INT8, path_out);
}

ql_status moe_int4(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint16_t* router_logits,
                   const int32_t* topk_ids_in, const float* topk_w_in, int E, int topk, int renormalize,
                   const uint8_t* w13, int64_t ldw13, int64_t w_estride13, const uint16_t* s13, int64_t lds13,
                   int64_t s_estride13, const uint8_t* z13, int64_t ldz13, int64_t z_estride13, const uint8_t* w2,
                   int64_t ldw2, int64_t w_estride2, const uint16_t* s2, int64_t lds2, int64_t s_estride2,
                   const uint8_t* z2, int64_t ldz2, int64_t z_estride2, int scale_fmt, int64_t group, int64_t I,
                   float swiglu_alpha, float swiglu_limit, int32_t* topk_ids_out, float* topk_w_out,
                   uint16_t* h_out, uint16_t* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                   ql_stream_t stream, int* path_out) {
  if (path_out) *path_out = QL_PATH_NONE;
  const Moe a = {x, M, H, ldx, router_logits, topk_ids_in, topk_w_in, E, topk, renormalize, I, swiglu_alpha,
                 swiglu_limit, topk_ids_out, topk_w_out, h_out, y, ldy, workspace, workspace_bytes};
  const Matrix a13 = {w13, ldw13, w_estride13}, a2 = {w2, ldw2, w_estride2};
  if (!s13 || !s2 || group < 1 || (scale_fmt != QL_SCALE_BF16 && scale_fmt != QL_SCALE_FP16)) return QL_ERR_INVALID_ARG;
  if (const ql_status s = moe_check(a, a13, a2, 32, 1); s != QL_OK) return s;
  if (lds13 < cdiv(H, group) || lds2 < cdiv(I, group) || s_estride13 < 0 || s_estride2 < 0) return QL_ERR_INVALID_ARG;
  if ((z13 && (ldz13 < cdiv(H, group) || z_estride13 < 0)) || (z2 && (ldz2 < cdiv(I, group) || z_estride2 < 0)))
    return QL_ERR_INVALID_ARG;
  if (group < 32 || (group & (group - 1)) != 0 || group > (1 << 28)) return QL_ERR_UNSUPPORTED;
  if (!aligned<2>(s13) || !aligned<2>(s2)) return QL_ERR_ALIGNMENT;
  StreamArgs gu = moe_args(a), dn = gu;
  gu.scale = s13;
  gu.lds = lds13;
  gu.s_estride = s_estride13;
  gu.zero = z13;
  gu.ldz = ldz13;
  gu.z_estride = z_estride13;
  dn.scale = s2;
  dn.lds = lds2;
  dn.s_estride = s_estride2;
  dn.zero = z2;
  dn.ldz = ldz2;
  dn.z_estride = z_estride2;
  gu.scale_fp16 = dn.scale_fp16 = scale_fmt == QL_SCALE_FP16;
  while ((int64_t(1) << gu.group_shift) < group) ++gu.group_shift;
  dn.group_shift = gu.group_shift;
  return moe_run(STREAM_INT4, a, a13, a2, gu, dn, (cudaStream_t)stream, QL_PATH_MOE_INT4, path_out);
}

}  // extern "C"
