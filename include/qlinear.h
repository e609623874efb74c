/*
 * qlinear.h - C ABI of the GB300 (sm_103a) quantized decode linear layer.
 *
 * Three weight formats of the decode-time weight-quantized linear layer (skinny GEMM,
 * M = 1..256 tokens), as described by the two source pages:
 *   [Z100] "Hygon Z100 (gfx906) vLLM adaptation: full record of optimisation and operator
 *          development (condensed)", chapter 二 (self-written operators) and chapter 三 §2;
 *   [DSV4] "vLLM 0.27.x port: DeepSeek V4 Flash FP4 on Hygon DCU - full report".
 *
 * Conventions shared by every entry point
 *   - Every tensor pointer is a DEVICE pointer (cudaMalloc / PyTorch CUDA memory) owned by
 *     the caller; the library never allocates, frees or synchronises, and enqueues all work
 *     on `stream` (a cudaStream_t; NULL = the legacy default stream).
 *   - bf16 tensors are passed as uint16_t bit patterns; fp8 E4M3, packed fp4 E2M1 and
 *     UE8M0 scales as uint8_t bytes.  All matrices are row-major with an explicit leading
 *     dimension (elements for bf16/int8/fp8, BYTES for packed fp4).
 *   - Every argument is validated on the host before any launch.  An invalid call returns
 *     an error status and launches nothing: no device assert, no silent copy ([Z100] §二.2.4
 *     "non-unit inner stride is an explicit error"; [Z100] chapter 四 on skinny kernels that
 *     device-asserted on unsupported sizes).
 *   - `workspace` is caller-owned device scratch of at least ql_workspace_bytes(...) bytes,
 *     16-byte aligned.  It must be zeroed once after allocation (ql_workspace_init); the
 *     kernels leave it reusable.  Calls that share a workspace must not overlap in time.
 *   - `path_out` (nullable HOST pointer) receives the QL_PATH_* code of the kernel sequence
 *     that ran: a dispatch marker, so tests can assert which path was taken.
 *   - Kernels that wait on barriers bound every wait; a wait that runs out sets a flag in
 *     the workspace status word (read it with ql_read_device_status) and the kernel exits
 *     cleanly.  Such a call's outputs are undefined.
 */
#ifndef QLINEAR_H
#define QLINEAR_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define QL_API __attribute__((visibility("default")))
#else
#define QL_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* ql_stream_t; /* identical to cudaStream_t */

typedef enum {
  QL_OK = 0,
  QL_ERR_INVALID_ARG = 1, /* null pointer, negative or inconsistent size            */
  QL_ERR_UNSUPPORTED = 2, /* valid but not implemented (shape, block size, mode)      */
  QL_ERR_ALIGNMENT = 3,   /* base pointer / leading dimension not 16-byte aligned     */
  QL_ERR_WORKSPACE = 4,   /* workspace null or smaller than ql_workspace_bytes()      */
  QL_ERR_CUDA = 5,        /* a CUDA runtime call failed (launch error)                */
  QL_ERR_TIMEOUT = 6      /* a bounded device-side wait ran out (ql_read_device_status)*/
} ql_status;

/* operation ids for ql_workspace_bytes */
enum { QL_OP_INT8_W8A8 = 1, QL_OP_FP8_BLOCK = 2, QL_OP_MXFP4 = 3, QL_OP_MOE_MXFP4 = 4, QL_OP_BF16 = 5,
       QL_OP_FP8_CHANNEL = 6, QL_OP_GATED_FFN = 7, QL_OP_GATED_FFN_BWD = 8, QL_OP_INT8_CODES = 9,
       QL_OP_MOE_FEW = 10 };

/* scale formats of the 4-bit group-scaled weights */
enum { QL_SCALE_BF16 = 0, QL_SCALE_FP16 = 1 };

/* what gated_ffn keeps of g and u for gated_ffn_backward */
enum { QL_SAVE_NONE = 0, QL_SAVE_BF16 = 1, QL_SAVE_INT8 = 2 };

/* output types of qlinear_int8 */
enum { QL_OUT_BF16 = 0, QL_OUT_FP16 = 1, QL_OUT_FP32 = 2 };

/* FP8 weight code formats of qlinear_fp8 */
enum { QL_FP8_E4M3 = 0 /* e4m3fn: bias 7, no infinities, S.1111.111 is NaN */,
       QL_FP8_E5M2 = 1 /* e5m2: bias 15, IEEE-style infinities and NaNs      */ };

/* activation modes of the FP8-block and MXFP4 linears */
enum {
  QL_ACT_BF16 = 0,      /* bf16 activations used as they are (a_s = 1)                        */
  QL_ACT_E4M3_1X128 = 1 /* activations quantised per token and per 128-K group to E4M3 with a
                           UE8M0 power-of-two scale (smallest 2^e with amax <= 448*2^e),
                           [DSV4] §3.3 quant_config "activation_scheme: dynamic, fmt e4m3,
                           scale_fmt ue8m0"                                                   */
};

/* dispatch markers written to *path_out */
enum {
  QL_PATH_NONE = 0,
  QL_PATH_INT8_SKINNY = 1,     /* skinny tensor-core GEMM, per-token INT8 quant in the launch */
  QL_PATH_FP8_SKINNY = 2,      /* FP8 block skinny GEMM, bf16 activations                   */
  QL_PATH_FP8_TCGEN05 = 3,     /* 1x128 act quant + tcgen05 block-scaled GEMM (FP8 x FP8)   */
  QL_PATH_MXFP4_SKINNY = 4,    /* MXFP4 skinny GEMM, bf16 activations                       */
  QL_PATH_MXFP4_TCGEN05 = 5,   /* 1x128 act quant + tcgen05 block-scaled GEMM (E4M3 x E2M1) */
  QL_PATH_MOE_MXFP4 = 6,       /* routing + dispatch + gate_up/SiLU + down + combine         */
  QL_PATH_BF16_SKINNY = 7,     /* BF16 skinny GEMM (unquantised weights)                    */
  QL_PATH_FP8_CHANNEL_SKINNY = 8, /* FP8 skinny GEMM, per-channel / per-tensor fp32 scale    */
  QL_PATH_INT8_TCGEN05 = 9,      /* per-token INT8 quant + tcgen05 GEMM on exact f16 images  */
  QL_PATH_MOE_MXFP4_TCGEN05 = 10, /* M > 16: routing + grouped tcgen05 GEMMs, 1x128 E4M3 act  */
  QL_PATH_INT4_SKINNY = 11,      /* 4-bit group-scaled skinny GEMM, bf16 activations         */
  QL_PATH_GATED_FFN_INT4 = 12,   /* gated block on 4-bit weights, one skinny launch           */
  QL_PATH_GATED_FFN_SKINNY = 13, /* gated block on bf16 weights, one skinny launch            */
  QL_PATH_GATED_FFN_TCGEN05 = 14, /* gated block, one tcgen05 GEMM with the activation in its epilogue */
  QL_PATH_GATED_FFN_BACKWARD = 15, /* gradients of g and u, then the dx and dW13 tcgen05 GEMMs */
  QL_PATH_INT8_CODES_SKINNY = 16,  /* given 8-bit codes, weight-streaming kernel                */
  QL_PATH_INT8_CODES_TCGEN05 = 17, /* given 8-bit codes, tcgen05 GEMM on pairs of SMs           */
  QL_PATH_MOE_BF16 = 18,           /* routing + gate, up and activation; down and the weighted  */
  QL_PATH_MOE_INT8 = 19,           /* sum: two weight-streaming launches                        */
  QL_PATH_MOE_INT4 = 20
};

/* device status flags (bitmask) */
enum { QL_DEV_TIMEOUT = 1u };

QL_API const char* ql_status_string(ql_status s);
QL_API int ql_version(void);

/*
 * Bytes of workspace the op needs for these sizes.  Every layout starts with the same
 * 256 + 1 MiB: the device status word and counters, then a region that is zero between calls
 * (split-K tickets, or the output cells of INT8 calls of up to 4 tokens), so one workspace can
 * serve calls of any op and shape in turn.  M, N, K as in the op; for
 * QL_OP_MOE_MXFP4: M tokens, N = H (hidden), K = I (expert intermediate), E experts and
 * topk routed experts per token.  QL_OP_GATED_FFN, QL_OP_GATED_FFN_BWD: N = I, K = H.  Returns 0 for an unknown op or negative sizes.
 */
QL_API size_t ql_workspace_bytes(int op, int64_t M, int64_t N, int64_t K, int E, int topk);

/* Zero `bytes` of workspace on `stream` (cudaMemsetAsync).  Call once after allocating. */
QL_API ql_status ql_workspace_init(void* workspace, size_t bytes, ql_stream_t stream);

/* Which CUDA graph capture `stream` takes part in (the capture's id; 0: none). */
QL_API uint64_t ql_capture_id(ql_stream_t stream);

/*
 * Read (and, if clear != 0, reset) the device status word of `workspace`; synchronises
 * `stream`.  *flags_out receives the QL_DEV_* bits.  Returns QL_ERR_TIMEOUT if the timeout
 * bit was set, QL_OK otherwise.  Test and debugging aid: the compute calls never read it.
 */
QL_API ql_status ql_read_device_status(void* workspace, ql_stream_t stream, int clear, uint32_t* flags_out);

/*
 * Iteration cap of every bounded device wait (default 1<<20 polls).  A test knob: a small
 * cap makes waits run out so the timeout path can be exercised without a hung GPU.
 */
QL_API void ql_set_wait_limit(uint32_t polls);

/*
 * INT8 W8A8 linear with dynamic per-token activation quantisation
 * ([Z100] §二.2 operator table "INT8 W8A8 sdot4" and §二.2.1):
 *   x_s[m]  = max_k |x[m,k]| / 127                       (fp32 IEEE division)
 *   x_q[m,k]= clamp(round_half_even(x[m,k] / x_s[m]), -127, 127)   (0 if x_s == 0)
 *   acc[m,n]= sum_k x_q[m,k] * w[n,k]                    (exact int32)
 *   y[m,n]  = bf16((acc * x_s[m]) * w_s[n])  then, if bias, y = bf16(y + bias[n])
 * x: bf16 [M, ldx] (K used); w: int8 [N, ldw], K-contiguous, used as stored (no transpose,
 * no dequantised copy); w_scale: fp32 [N] (per channel) or [1] (per tensor, w_scale_len == 1);
 * bias: nullable bf16 [N]; y: bf16 [M, ldy].
 * Debug outputs (nullable): acc_out int32 [M, N] (dense, ld N), xq_out int8 [M, K] (ld K),
 * xs_out fp32 [M].
 * Paths: M <= 32 -> the persistent skinny kernel (quantisation fused in, one launch);
 *        M > 32  -> a quantisation launch + the tcgen05 GEMM (kind::f16 MMAs on the exact f16
 *                   values of the codes and weights, drained to int32 every 512 K).
 * Requires: M >= 1, N >= 1, K >= 16, K % 16 == 0, ldx >= K, ldw >= K, ldw % 16 == 0,
 * ldy >= N, 16-byte aligned x and w, |acc| < 2^31 (always true for K <= 133152).
 */
QL_API ql_status qlinear_int8_w8a8(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                            const int8_t* w, int64_t N, int64_t ldw,
                            const float* w_scale, int64_t w_scale_len,
                            const uint16_t* bias, uint16_t* y, int64_t ldy,
                            int32_t* acc_out, int8_t* xq_out, float* xs_out,
                            void* workspace, size_t workspace_bytes, ql_stream_t stream,
                            int* path_out);

/*
 * FP8 E4M3 weights with block UE8M0 scales ([Z100] §二.2.4 "block-scaled (128x128) FP8
 * extension"; chapter 三 §2):
 *   y[m,n] = bf16( sum_kb a_s[m,kb] * 2^(w_scale[n/block_n, kb] - 127)
 *                        * sum_{k in kb} a[m,k] * e4m3(w[n,k]) )   (+ bias after the cast)
 * act_mode QL_ACT_BF16: a = x (bf16), a_s = 1.  QL_ACT_E4M3_1X128: a = e4m3 codes and a_s
 * their UE8M0 scales from the 1x128 quantisation of x (block_k must then be 128).
 * x: bf16 [M, ldx]; w: E4M3 bytes [N, ldw] (padded rows allowed, e.g. ldw = K + 256);
 * w_scale: UE8M0 [ceil(N/block_n), ceil(K/block_k)] row-major; y: bf16 [M, ldy].
 * Debug outputs (nullable, act_mode 1 only): aq_out E4M3 [M, K], as_out UE8M0 [M, ceil(K/128)].
 * Paths: act_mode 0 -> skinny tensor-core kernel (block_n % 16 == 0, block_k % 64 == 0);
 *        act_mode 1 -> tcgen05 block-scaled GEMM (block_n == block_k == 128).
 * Requires K % 16 == 0 (act_mode 1: K % 128 == 0), ldw % 16 == 0, 16-byte aligned x and w.
 */
QL_API ql_status qlinear_fp8_block(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                            const uint8_t* w, int64_t N, int64_t ldw,
                            const uint8_t* w_scale, int block_n, int block_k, int act_mode,
                            const uint16_t* bias, uint16_t* y, int64_t ldy,
                            uint8_t* aq_out, uint8_t* as_out,
                            void* workspace, size_t workspace_bytes, ql_stream_t stream,
                            int* path_out);

/*
 * MXFP4 weights: E2M1 codes packed two per byte (element 2i in the LOW nibble of byte i)
 * with one UE8M0 scale per 32 consecutive K elements of a row ([DSV4] §9.3, MXFP4 expert
 * weights kept in checkpoint format and dequantised on demand):
 *   y[m,n] = bf16( sum_k a[m,k] * e2m1(w[n,k]) * 2^(w_scale[n, k/32] - 127) ) (+ bias)
 * act_mode QL_ACT_BF16: a = x.  QL_ACT_E4M3_1X128: a = e4m3(q[m,k]) * 2^(s[m,k/128]-127).
 * w: [N, ldw_bytes] (K/2 bytes used); w_scale: [N, lds] (K/32 used).
 * Paths: act_mode 0 -> skinny tensor-core kernel; act_mode 1 -> tcgen05 GEMM.
 * Requires K % 32 == 0 (act_mode 1: K % 128 == 0), ldw_bytes % 16 == 0, 16-byte aligned
 * x and w, lds >= K/32 (act_mode 1: lds % 16 == 0 and 16-byte aligned w_scale).
 */
QL_API ql_status qlinear_mxfp4(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                        const uint8_t* w, int64_t N, int64_t ldw_bytes,
                        const uint8_t* w_scale, int64_t lds, int act_mode,
                        const uint16_t* bias, uint16_t* y, int64_t ldy,
                        uint8_t* aq_out, uint8_t* as_out,
                        void* workspace, size_t workspace_bytes, ql_stream_t stream,
                        int* path_out);

/*
 * FP8 weights with one fp32 scale per output channel or per tensor ([Z100] §二.2.2, the
 * emulated FP8 GEMV: e4m3fn or e5m2 codes widened exactly, the scale applied once to the
 * finished dot product):
 *   y[m,n] = bf16( w_scale[n or 0] * sum_k x[m,k] * fp8(w[n,k]) ) (+ bias, added after the
 *   cast and rounded again)
 * x: bf16 [M, ldx] (device); w: FP8 codes [N, ldw] (device, K used, padded rows allowed);
 * w_fmt: QL_FP8_E4M3 or QL_FP8_E5M2; w_scale: fp32 [w_scale_len] (device), w_scale_len = N
 * (per channel) or 1 (per tensor); bias: bf16 [N] or null; y: bf16 [M, ldy] (device).  The
 * caller owns every buffer; nothing is retained after the call returns.  Codes must be finite
 * (NaN / infinity codes propagate through the sum).  Runs the persistent skinny kernel 16
 * tokens at a time, bf16 activations.
 * Requires K % 16 == 0, ldx % 8 == 0, ldw % 16 == 0, 16-byte aligned x and w, ldy >= N;
 * returns QL_ERR_INVALID_ARG / QL_ERR_ALIGNMENT / QL_ERR_UNSUPPORTED before any launch
 * otherwise.  workspace: ql_workspace_bytes(QL_OP_FP8_CHANNEL, M, N, K, 0, 0) bytes, zeroed once.
 */
QL_API ql_status qlinear_fp8(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                      const uint8_t* w, int64_t N, int64_t ldw, int w_fmt,
                      const float* w_scale, int64_t w_scale_len,
                      const uint16_t* bias, uint16_t* y, int64_t ldy,
                      void* workspace, size_t workspace_bytes, ql_stream_t stream,
                      int* path_out);

/*
 * BF16 dense decode GEMV, unquantised weights ([Z100] §二.2.3, the bf16 route: bf16 widened to
 * fp32 exactly, products summed in fp32):
 *   y[m,n] = bf16( sum_k x[m,k] * w[n,k] ) (+ bias, added after the cast and rounded again)
 * x: bf16 [M, ldx] (device), w: bf16 [N, ldw] (device, K used, padded rows allowed), bias:
 * bf16 [N] or null, y: bf16 [M, ldy] (device).  The caller owns every buffer; nothing is
 * retained after the call returns.  Runs the persistent skinny kernel 16 tokens at a time.
 * Requires K % 8 == 0, ldx % 8 == 0, ldw % 8 == 0, 16-byte aligned x and w, ldy >= N; returns
 * QL_ERR_INVALID_ARG / QL_ERR_ALIGNMENT / QL_ERR_UNSUPPORTED before any launch otherwise.
 * workspace: ql_workspace_bytes(QL_OP_BF16, M, N, K, 0, 0) bytes, zeroed once.
 */
QL_API ql_status qlinear_bf16(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                       const uint16_t* w, int64_t N, int64_t ldw, const uint16_t* bias,
                       uint16_t* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                       ql_stream_t stream, int* path_out);

/*
 * MXFP4 mixture-of-experts decode layer ([DSV4] §0.1 "M=1 MoE routing Q1", §0.3 grouped
 * batch MoE, §9.3 MXFP4 emulation experts):
 *   routing : p = softmax(router_logits[m, :E]); ids = the topk largest logits (ties go to
 *             the lower expert id), ordered by decreasing logit; weights = p[ids]
 *             (divided by their sum if renormalize != 0).  Alternatively the caller passes
 *             topk_ids_in / topk_w_in and router_logits = NULL (exactly one of the two).
 *             The weights are fp32 exponentials over a float-float sum: within a few fp32
 *             ulps of the exact softmax; the ids depend on logit comparisons only.
 *   dispatch: (token, slot) pairs grouped by expert, pairs of one expert in pair order.
 *   gate_up : for pair (m,j) with expert e: g = W13[e][0:I] x_m, u = W13[e][I:2I] x_m,
 *             h = bf16( silu(alpha * min(g, limit)) * clamp(u, -limit, limit) )
 *             (the clamped SwiGLU of [DSV4] §6.6 / §9.4, alpha = swiglu_alpha, limit =
 *             swiglu_limit; limit = +infinity with alpha = 1 is the plain silu(g) * u)
 *   down    : y[m] = bf16( sum_j weight[m,j] * W2[e_(m,j)] h_(m,j) )
 * x: bf16 [M, H]; router_logits: bf16 [M, E]; topk_ids_in int32 [M, topk];
 * topk_w_in fp32 [M, topk]; w13: [E, 2I, H/2] packed E2M1, s13: [E, 2I, H/32] UE8M0;
 * w2: [E, H, I/2], s2: [E, H, I/32]; y: bf16 [M, H] (dense).
 * Debug outputs (nullable): topk_ids_out int32 [M, topk], topk_w_out fp32 [M, topk],
 * h_out bf16 [M*topk, I] (row m*topk + j).
 * swiglu_alpha must be finite; swiglu_limit >= 0 (+infinity allowed), else QL_ERR_INVALID_ARG.
 * Paths: M <= 16: the persistent skinny kernel with bf16 activations (routing fused into the
 *        gate_up launch), QL_PATH_MOE_MXFP4; 9..16 tokens run as two such calls, tokens
 *        [0, 8) and [8, M) (tokens are independent; one 8-token tile per call is cheaper);
 *        M > 16: grouped tcgen05 GEMMs over the routed experts ([DSV4] §0.3 grouped batch MoE),
 *        QL_PATH_MOE_MXFP4_TCGEN05: x and h are quantised per token and 128-K group to E4M3 with
 *        a UE8M0 scale before their GEMMs (the activation format of qlinear_mxfp4's act_mode 1).
 * Requires 1 <= M <= 65535, 1 <= topk <= min(E, 16), E <= 1024, H % 128 == 0, I % 128 == 0,
 * 16-byte aligned weight pointers.
 */
QL_API ql_status moe_mxfp4_grouped(const uint16_t* x, int64_t M, int64_t H,
                            const uint16_t* router_logits, const int32_t* topk_ids_in,
                            const float* topk_w_in, int E, int topk, int renormalize,
                            const uint8_t* w13, const uint8_t* s13,
                            const uint8_t* w2, const uint8_t* s2, int64_t I,
                            float swiglu_alpha, float swiglu_limit,
                            int32_t* topk_ids_out, float* topk_w_out, uint16_t* h_out,
                            uint16_t* y, void* workspace, size_t workspace_bytes,
                            ql_stream_t stream, int* path_out);

/*
 * Sharded (tensor-parallel) layers.  The pages run these linears split over 2, 4 or 8 GPUs
 * ([Z100] chapter 一 §5, communication and parallelism under TP = 2/4/8; [DSV4] §0, TP = 4/8):
 *   - column-parallel (N split): every shard is a plain call of the entry points above on its
 *     rows of W (FP8 block scales: shard boundaries on whole block_n rows); the concatenated
 *     outputs are the unsharded layer's outputs, bit for bit.
 *   - row-parallel (K split): every shard holds a K range of W and of x (FP8 block: whole
 *     block_k ranges; MXFP4: whole 256-K units, so its scale rows stay whole bytes per shard).
 *     INT8: each shard's ql_token_amax, an all-reduce MAX across shards, then
 *     qlinear_int8_w8a8_partial on each shard with that amax (its codes are then exactly the
 *     unsharded codes), an all-reduce SUM of the int32 sums (exact) and qlinear_int8_epilogue:
 *     the result equals the unsharded call's bit for bit.  FP8 / MXFP4: each shard's fp32
 *     partial sums (the *_partial entry points), an all-reduce SUM, then ql_finish_f32 rounds
 *     once to bf16 and adds the bias.  The collectives are the caller's (NCCL, gloo, ...).
 * Pointers are device pointers owned by the caller; nothing is allocated or retained.
 */

/* Per-token amax of a K shard: amax_out[m] = max_k |x[m,k]| (fp32 [M]).  K % 8 == 0,
 * 16-byte aligned x, ldx % 8 == 0. */
QL_API ql_status ql_token_amax(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, float* amax_out,
                               ql_stream_t stream);

/* A K shard of a row-parallel INT8 W8A8 layer: x_s[m] = amax[m] / 127 (amax: the tokens'
 * amax over the whole row, fp32 [M]), codes as in qlinear_int8_w8a8, and the exact int32
 * sums over this shard's K written to acc_out [M, N] (dense, required); no epilogue, no y.
 * xq_out (nullable) receives the codes.  Same requirements and workspace as
 * qlinear_int8_w8a8. */
QL_API ql_status qlinear_int8_w8a8_partial(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                           const int8_t* w, int64_t N, int64_t ldw, const float* amax,
                                           int32_t* acc_out, int8_t* xq_out, void* workspace,
                                           size_t workspace_bytes, ql_stream_t stream, int* path_out);

/* The INT8 epilogue on int32 sums added over the shards: y = bf16((acc * x_s) * w_s) (+ bias
 * after the cast), x_s = amax / 127 (IEEE fp32 division), acc int32 [M, N] dense. */
QL_API ql_status qlinear_int8_epilogue(const int32_t* acc, int64_t M, int64_t N, const float* amax,
                                       const float* w_scale, int64_t w_scale_len, const uint16_t* bias,
                                       uint16_t* y, int64_t ldy, ql_stream_t stream);

/* A K shard of a row-parallel FP8-block layer (bf16 activations): y32[m,n] = the fp32 sum of
 * this shard's scaled block products (no bias), [M, ldy32].  block_k a power of two >= 64,
 * block_n % 16 == 0; otherwise as qlinear_fp8_block with act_mode QL_ACT_BF16. */
QL_API ql_status qlinear_fp8_block_partial(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                           const uint8_t* w, int64_t N, int64_t ldw, const uint8_t* w_scale,
                                           int block_n, int block_k, float* y32, int64_t ldy32,
                                           void* workspace, size_t workspace_bytes, ql_stream_t stream,
                                           int* path_out);

/* A K shard of a row-parallel MXFP4 layer (bf16 activations): fp32 partial sums into y32
 * [M, ldy32], no bias.  K % 256 == 0, lds % 8 == 0 and 8-byte aligned w_scale (else
 * QL_ERR_UNSUPPORTED); otherwise as qlinear_mxfp4 with act_mode QL_ACT_BF16. */
QL_API ql_status qlinear_mxfp4_partial(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                       const uint8_t* w, int64_t N, int64_t ldw_bytes, const uint8_t* w_scale,
                                       int64_t lds, float* y32, int64_t ldy32, void* workspace,
                                       size_t workspace_bytes, ql_stream_t stream, int* path_out);

/* One bf16 rounding of fp32 sums added over the shards, then + bias (after the cast, rounded
 * again): y[m,n] = bf16(bf16(y32[m,n]) + bias[n]). */
QL_API ql_status ql_finish_f32(const float* y32, int64_t M, int64_t N, int64_t ld32, const uint16_t* bias,
                               uint16_t* y, int64_t ldy, ql_stream_t stream);

/*
 * INT8 W8A8 linear that allocates nothing and takes no workspace.  The pages have no
 * counterpart: this entry point exists for callers that cannot give the library device
 * memory - hosts without a device allocator of their own, plugins inside a framework that
 * has reserved all GPU memory for its pool and forbids new cudaMalloc calls, and latency-
 * critical paths that must not call cudaMalloc/cudaFree because those can synchronise the
 * device.  It computes exactly what qlinear_int8_w8a8 computes (same arguments, minus the
 * workspace) and takes its scratch from a 16 MiB array in the library's own device memory,
 * held on every GPU that loads the library until the process exits.
 *   - The first call on each device looks up that array's device address (with the device
 *     current) and caches it; make that first call before any stream capture.
 *   - Sizes whose scratch need (ql_workspace_bytes(QL_OP_INT8_W8A8, M, N, K, 0, 0)) exceeds
 *     16 MiB are rejected with QL_ERR_WORKSPACE; nothing is launched.
 *   - All calls on a device share the array: each call clears what must start at zero on its
 *     stream, and calls that overlap on the GPU (unordered streams) race on it.
 *   - It never calls cudaMalloc, cudaFree or any allocating routine.
 */
QL_API ql_status qlinear_int8_w8a8_noalloc(const uint16_t* x, int64_t M, int64_t K, int64_t ldx,
                                           const int8_t* w, int64_t N, int64_t ldw,
                                           const float* w_scale, int64_t w_scale_len,
                                           const uint16_t* bias, uint16_t* y, int64_t ldy,
                                           int32_t* acc_out, int8_t* xq_out, float* xs_out,
                                           ql_stream_t stream, int* path_out);

/*
 * Linear layer on 4-bit integer weights with one scale (and zero point) per group of K
 * elements of a row:
 *   w[n,k] = (q[n,k] - z[n,k/group]) * s[n,k/group]
 *   y[m,n] = bf16( sum_k x[m,k] * w[n,k] )  then, if bias, y = bf16(y + bias[n])
 * q: codes 0..15 packed two per byte, element 2i in the LOW nibble of byte i, rows of
 * ldw_bytes; s: bf16 (QL_SCALE_BF16) or fp16 (QL_SCALE_FP16) bits [N, lds], lds >=
 * ceil(K/group), |s| < 2^122; z: uint8 [N, ldz], or NULL for 8 everywhere (symmetric
 * codes);
 * x: bf16 [M, ldx]; bias: nullable bf16 [N]; y: bf16 [M, ldy].  q - z is exact in bf16, its
 * products with x are exact in fp32 and every group's fp32 sum is multiplied by its scale once:
 * no weight is rounded.  Weights are streamed once per 32 tokens.
 * Requires: 1 <= M <= 65535, K % 32 == 0 (the last group may be short), group a power of two
 * >= 32 (a group >= K is one scale per row), ldx >= K, ldx % 8 == 0, ldw_bytes >= K/2,
 * ldw_bytes % 16 == 0, 16-byte aligned x and w, 2-byte aligned scales, bias and y, ldy >= N.
 * Takes no workspace and waits on nothing inside the kernel.
 */
QL_API ql_status qlinear_int4(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint8_t* w, int64_t N,
                              int64_t ldw_bytes, const uint16_t* w_scale, int scale_fmt, int64_t lds,
                              const uint8_t* w_zero, int64_t ldz, int64_t group, const uint16_t* bias, uint16_t* y,
                              int64_t ldy, ql_stream_t stream, int* path_out);

/*
 * Gated feed-forward block: both projections, the activation and the product in one launch.
 *   g[m,i] = sum_k x[m,k] W13[i,k],  u[m,i] = sum_k x[m,k] W13[I+i,k]      (fp32)
 *   h[m,i] = bf16( silu(alpha * min(g, limit)) * clamp(u, -limit, limit) )
 * (moe_mxfp4_grouped's expert activation; limit = +infinity with alpha = 1 is silu(g) * u.)
 * x: bf16 [M, ldx] (H used); w13: bf16 [2I, ldw], rows [0, I) gate and [I, 2I) up; h: bf16
 * [M, ldh].
 * save != QL_SAVE_NONE keeps g and u for gated_ffn_backward in ckpt, two halves per token, each
 * of P = I rounded up to 128 columns: QL_SAVE_BF16: bf16 [M, 2, P]; QL_SAVE_INT8: int8
 * [M, 2, P] and ckpt_scale fp32 [M, 2, P/128], per token and 128 columns
 *   scale = max|v| / 127,  code = round_half_even(v * (127 / max|v|)), all in fp32: within 2^-16 of a
 * tie it may be the other neighbour of v / scale  (scale 0 where max|v| < 2^-100; an infinity or a
 * NaN in a group reads back as NaN throughout it).  Columns I..P are
 * undefined.
 * Paths: without a checkpoint, M <= 16, or more where ceil(M/32) ceil(I/16) is at most four times
 *        (M <= 32) or twice the number of SMs: a skinny launch that streams the weights once per 32
 *        tokens; else one tcgen05 GEMM whose epilogue applies the activation and writes h and the checkpoint.
 * Requires: 1 <= M <= 2^22, H and I multiples of 8, at most 2^20, ldx >= H, ldw >= H, ldh >= I,
 * leading dimensions multiples of 8, 16-byte aligned x, w13, h and ckpt, 4-byte aligned ckpt_scale;
 * alpha finite, limit >= 0.  workspace: ql_workspace_bytes(QL_OP_GATED_FFN, M, I, H, 0, 0) bytes,
 * zeroed once.  Outputs of a call that raised QL_DEV_TIMEOUT in its status word are incomplete; the
 * next call needs nothing.
 */
QL_API ql_status gated_ffn(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint16_t* w13, int64_t I,
                           int64_t ldw, float swiglu_alpha, float swiglu_limit, uint16_t* h, int64_t ldh, int save,
                           void* ckpt, float* ckpt_scale, void* workspace, size_t workspace_bytes,
                           ql_stream_t stream, int* path_out);

/*
 * The block's backward pass from the checkpoint of its forward (save QL_SAVE_BF16 or
 * QL_SAVE_INT8; G and U are the values that the checkpoint stands for), with g' = min(G, limit)
 * and u' = clamp(U, -limit, limit):
 *   du = dh * silu(alpha g') where |U| <= limit, else 0
 *   dg = dh * u' * alpha * silu'(alpha g') where G <= limit, else 0
 *   dx = bf16( dg W13[0:I] + du W13[I:2I] ),  dw13 = bf16( [dg du]^T x )
 * dg and du are rounded to bf16 (the tensor cores' operands: dx and dw13 are then 0.0024 of their
 * norm from exact, 0.0017 of it the outputs' own rounding), the sums are fp32.  dh: bf16
 * [M, ld_dh]; x, w13 as in the forward; dx: bf16 [M, ld_dx] or NULL; dw13: bf16 [2I, ld_dw] or
 * NULL (one of the two is required; x is not read without dw13, w13 not without dx).
 * Deterministic: the same sizes and the same set of outputs are summed in the same order, whatever
 * runs when.  A gradient alone may be summed in another order than together with the other one.
 * Requires what gated_ffn requires, ld_dh >= I, ld_dx >= H, ld_dw >= H (multiples of 8) and
 * 16-byte aligned dh, dx, dw13.  workspace: ql_workspace_bytes(QL_OP_GATED_FFN_BWD, M, I, H, 0, 0)
 * bytes (it holds [dg du]), zeroed once.
 */
QL_API ql_status gated_ffn_backward(const uint16_t* dh, int64_t ld_dh, const uint16_t* x, int64_t M, int64_t H,
                                    int64_t ldx, const uint16_t* w13, int64_t I, int64_t ldw, float swiglu_alpha,
                                    float swiglu_limit, int save, const void* ckpt, const float* ckpt_scale,
                                    uint16_t* dx, int64_t ld_dx, uint16_t* dw13, int64_t ld_dw, void* workspace,
                                    size_t workspace_bytes, ql_stream_t stream, int* path_out);

/*
 * How the block's GEMMs are laid out for these sizes (no launch): what the tests of the split paths
 * check their shapes by.  gemm: QL_FFN_GEMM_FORWARD (mode: QL_SAVE_*), _DX or _DW (mode: 1 if the
 * call computes both gradients, 0 if this one alone).  out receives
 *   [0] pairs of CTAs that share the GEMM (0: the few-token kernel, and the rest 0)
 *   [1] columns of a tile   [2] tiles taken whole
 *   [3] tiles after them that are cut along the summed dimension, [4] each into so many parts
 *   [5] launches that the call's GEMMs take (both gradients: 1 side by side, 2 one after the other)
 */
enum { QL_FFN_GEMM_FORWARD = 0, QL_FFN_GEMM_DX = 1, QL_FFN_GEMM_DW = 2 };
QL_API ql_status ql_gated_ffn_plan(int gemm, int64_t M, int64_t I, int64_t H, int mode, int32_t* out);

/*
 * The gated block's form for few tokens on 4-bit weights: w13's 2I rows are stored, scaled and
 * required as qlinear_int4's (K = H), h and the activation are as gated_ffn's.  g and u stay in
 * fp32.  One launch per call, no workspace.
 */
QL_API ql_status gated_ffn_int4(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint8_t* w13, int64_t I,
                                int64_t ldw_bytes, const uint16_t* w_scale, int scale_fmt, int64_t lds,
                                const uint8_t* w_zero, int64_t ldz, int64_t group, float swiglu_alpha,
                                float swiglu_limit, uint16_t* h, int64_t ldh, ql_stream_t stream, int* path_out);

/*
 * 8-bit codes of tokens, by the rule of qlinear_int8_w8a8, for projections that share them:
 *   scale[m] = max_k |x[m,k]| / 127,  codes[m,k] = clamp(round_half_even(x[m,k] / scale[m]), -127, 127)
 * (IEEE fp32 divisions; an all-zero token has scale 0 and codes 0; one with an infinity or a NaN has
 * that for its scale, and codes of no meaning.)  x: bf16 [M, ldx]; codes: int8
 * [M, K] dense; scale: fp32 [M].
 * Requires 1 <= M <= 2^22, K >= 8, K % 8 == 0, K <= 2^20, ldx >= K, ldx % 8 == 0, 16-byte aligned x
 * and codes.
 */
QL_API ql_status quantize_int8(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int8_t* codes, float* scale,
                               ql_stream_t stream);

/*
 * Linear layer on 8-bit codes on both sides, their scales given:
 *   acc[m,n] = sum_k x_q[m,k] * w[n,k]  (exact int32),  y[m,n] = out((acc * x_scale[m]) * w_scale[n])
 * then, if bias, y = out(y + bias[n]).  With quantize_int8's codes and scales of finite tokens and
 * QL_OUT_BF16 it is qlinear_int8_w8a8's y bit for bit (a token with a NaN: NaN throughout here, left out of
 * the largest magnitude there).  x_q: int8 [M, ldx]; x_scale: fp32 [M]; w: int8 [N, ldw], both of
 * any value, -128 too; w_scale: fp32 [N] or [1] (w_scale_len); bias: nullable bf16 [N]; y: [M, ldy] of
 * out_type QL_OUT_*.
 * Paths: M <= 16, or up to 1024 tokens on weights small enough: one launch that streams the weights once per
 *        16 tokens; else a launch that widens the tokens' codes to f16 and one tcgen05 GEMM that widens
 *        the weights on the way (sm_103a has no integer tcgen05 MMA; fp32 sums are exact below 2^24 and
 *        move to int32 every 1024 k).  The result is the same.
 * Requires 1 <= M <= 2^22, 1 <= N <= 2^24, K >= 16, K % 16 == 0, K <= 131056 (|acc| < 2^31), ldx >= K,
 * ldw >= K, both multiples of 16, 16-byte aligned x_q and w, 4-byte aligned scales, y aligned to its
 * type, ldy >= N.  workspace: ql_workspace_bytes(QL_OP_INT8_CODES, M, N, K, 0, 0) bytes, zeroed once.
 */
QL_API ql_status qlinear_int8(const int8_t* x_q, int64_t M, int64_t K, int64_t ldx, const float* x_scale,
                              const int8_t* w, int64_t N, int64_t ldw, const float* w_scale, int64_t w_scale_len,
                              const uint16_t* bias, int out_type, void* y, int64_t ldy, void* workspace,
                              size_t workspace_bytes, ql_stream_t stream, int* path_out);

/*
 * Mixture-of-experts layers for a few tokens on bf16, 8-bit and 4-bit weights: moe_mxfp4_grouped's
 * layer (routing, gate and up, activation, down, weighted sum; the same routing arguments, activation
 * and debug outputs) in two launches that stream every chosen expert's weights once per 8 of its
 * tokens.
 * Expert ids outside [0, E) are padding: the pair is left out, and a token without any expert gets
 * zeros (topk_ids_out reports -1, topk_w_out the weight as given, and the pair's row of h_out is zeros).
 *   h = bf16( silu(alpha * min(g, limit)) * clamp(u, -limit, limit) ),  y = bf16( sum_j weight_j W2[e_j] h_j )
 *   moe_bf16: w13 bf16 [E, 2I, H], w2 bf16 [E, H, I]; fp32 sums.
 *   moe_int8: w13 int8 [E, 2I, H] and s13 fp32 [E, 2I], w2 int8 [E, H, I] and s2 fp32 [E, H] (dense);
 *     x is quantised per token and h per pair by quantize_int8's rule (a row whose largest magnitude is
 *     below 2^-110 counts as zeros).  Gate and up are exact int32 sums.  Down is exact over runs of one expert's
 *     k, at most 1024 of them; a run is scaled and added to the token's sum in fp32, and where runs end
 *     (multiples of 128 k) depends on the call's sizes and routing.  A row with an infinity or a NaN gives
 *     NaN throughout.
 *   moe_int4: w13 packed codes [E, 2I, ldw13], w2 [E, H, ldw2] with scales and zero points stored as
 *     qlinear_int4's: s13 [E, 2I, lds13], s2 [E, H, lds2], z13, z2 likewise (each NULL: 8).  No weight
 *     is rounded; x and h stay bf16; a group's sum of (q - z) x is fp32 and meets its scale once.
 * Experts, rows and scale rows are ld / stride elements apart (packed codes: bytes): w_estride13 is the distance
 * of two experts of w13, and so on.  x: bf16 [M, ldx]; y: bf16 [M, ldy].
 * Requires 1 <= M <= 64, 1 <= topk <= min(E, 16), E <= 1024, H and I at most 32768 and multiples of 8
 * (bf16), 16 (int8), 32 (int4); 16-byte aligned x and weights, their rows and experts whole 16 bytes
 * apart; 4-byte aligned fp32 scales.  int4: one group for w13 and w2, a power of two >= 32.
 * workspace: ql_workspace_bytes(QL_OP_MOE_FEW, M, H, I, E, topk) bytes, zeroed once.
 */
QL_API ql_status moe_bf16(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint16_t* router_logits,
                          const int32_t* topk_ids_in, const float* topk_w_in, int E, int topk, int renormalize,
                          const uint16_t* w13, int64_t ldw13, int64_t w_estride13, const uint16_t* w2, int64_t ldw2,
                          int64_t w_estride2, int64_t I, float swiglu_alpha, float swiglu_limit,
                          int32_t* topk_ids_out, float* topk_w_out, uint16_t* h_out, uint16_t* y, int64_t ldy,
                          void* workspace, size_t workspace_bytes, ql_stream_t stream, int* path_out);
QL_API ql_status moe_int8(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint16_t* router_logits,
                          const int32_t* topk_ids_in, const float* topk_w_in, int E, int topk, int renormalize,
                          const int8_t* w13, int64_t ldw13, int64_t w_estride13, const float* s13, const int8_t* w2,
                          int64_t ldw2, int64_t w_estride2, const float* s2, int64_t I, float swiglu_alpha,
                          float swiglu_limit, int32_t* topk_ids_out, float* topk_w_out, uint16_t* h_out, uint16_t* y,
                          int64_t ldy, void* workspace, size_t workspace_bytes, ql_stream_t stream, int* path_out);
QL_API ql_status moe_int4(const uint16_t* x, int64_t M, int64_t H, int64_t ldx, const uint16_t* router_logits,
                          const int32_t* topk_ids_in, const float* topk_w_in, int E, int topk, int renormalize,
                          const uint8_t* w13, int64_t ldw13, int64_t w_estride13, const uint16_t* s13, int64_t lds13,
                          int64_t s_estride13, const uint8_t* z13, int64_t ldz13, int64_t z_estride13,
                          const uint8_t* w2, int64_t ldw2, int64_t w_estride2, const uint16_t* s2, int64_t lds2,
                          int64_t s_estride2, const uint8_t* z2, int64_t ldz2, int64_t z_estride2, int scale_fmt,
                          int64_t group, int64_t I, float swiglu_alpha, float swiglu_limit, int32_t* topk_ids_out,
                          float* topk_w_out, uint16_t* h_out, uint16_t* y, int64_t ldy, void* workspace,
                          size_t workspace_bytes, ql_stream_t stream, int* path_out);

#ifdef __cplusplus
}
#endif
#endif /* QLINEAR_H */
