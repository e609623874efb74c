// 8-bit codes and scales of bf16 tokens: scale = max|x| / 127 of the row, code = x / scale rounded half to
// even, by the fp32 divisions of the INT8 linear.
//
// A CTA takes a token and keeps it in registers between the two passes (V vectors of 8 values a thread),
// so that it is read once; longer rows are read again, from L2.  No value is divided: see code_factor.
// Bound by HBM and a CTA's two barriers: 4096 x 5120 (63 MB) 12 us, 5.2 TB/s; read twice and divided 24 us.
#include "common.cuh"
#include "ffn_act.cuh"
#include "internal.h"
#include "stream_dev.cuh"

namespace ql {

namespace {

constexpr int kThreads = 256;

// the low bytes of four whole numbers as floats: v f + 1.5 2^23 ends in the number's two's complement
__device__ __forceinline__ uint32_t codes4(uint32_t lo, uint32_t hi, float f) {
  auto one = [f](uint32_t bits) { return __float_as_uint(fmaf(__uint_as_float(bits), f, 12582912.f)); };
  const uint32_t a = __byte_perm(one(lo << 16), one(lo & 0xFFFF0000u), 0x0040);
  const uint32_t b = __byte_perm(one(hi << 16), one(hi & 0xFFFF0000u), 0x0040);
  return __byte_perm(a, b, 0x5410);
}

template <int V>
__global__ void __launch_bounds__(kThreads) token_codes_kernel(const uint16_t* __restrict__ x, int K, int64_t ldx,
                                                               int8_t* __restrict__ codes, float* __restrict__ scale) {
  __shared__ unsigned s_top[kThreads / 32];
  const int m = blockIdx.x, vecs = K / 8;
  pdl_wait();
  pdl_launch_dependents();
  const uint4* row = reinterpret_cast<const uint4*>(x + (int64_t)m * ldx);
  uint4 kept[V];
  float top = 0.f;
  auto take = [&](uint4 v) {
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      top = max_nan(max_nan(top, fabsf(__uint_as_float(q[j] << 16))), fabsf(__uint_as_float(q[j] & 0xFFFF0000u)));
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * kThreads + threadIdx.x;
    kept[i] = v < vecs ? row[v] : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) take(kept[i]);
  for (int v = V * kThreads + threadIdx.x; v < vecs; v += kThreads) take(row[v]);
  // as whole numbers: a NaN is above all
  const unsigned w = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7FFFFFFFu);
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = w;
  __syncthreads();
  unsigned most = 0u;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) most = max(most, s_top[i]);
  top = __uint_as_float(most);
  const float s = __fdiv_rn(top, 127.f), f = code_factor(top);
  if (threadIdx.x == 0) scale[m] = s;
  const bool tiny = f == 0.f && s > 0.f && top < 1.f;  // below 2^-110, where 127 / top is no number: divided
  uint2* out = reinterpret_cast<uint2*>(codes + (int64_t)m * K);
  auto put = [&](int v, uint4 q) {
    if (!tiny) {
      out[v] = make_uint2(codes4(q.x, q.y, f), codes4(q.z, q.w, f));
      return;
    }
    const uint32_t in[4] = {q.x, q.y, q.z, q.w};
    uint32_t packed[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xv = __uint_as_float(i & 1 ? in[i >> 1] & 0xFFFF0000u : in[i >> 1] << 16);
      const int c = (int)fminf(fmaxf(rintf(__fdiv_rn(xv, s)), -127.f), 127.f);
      packed[i >> 2] |= (uint32_t)(c & 0xFF) << (8 * (i & 3));
    }
    out[v] = make_uint2(packed[0], packed[1]);
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = i * kThreads + threadIdx.x;
    if (v < vecs) put(v, kept[i]);
  }
  for (int v = V * kThreads + threadIdx.x; v < vecs; v += kThreads) put(v, row[v]);
}

}  // namespace

cudaError_t launch_token_codes(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, int8_t* codes, float* scale,
                               cudaStream_t st) {
  const int64_t v = (K / 8 + kThreads - 1) / kThreads;
  auto* kfn = v <= 1 ? token_codes_kernel<1> : v <= 2 ? token_codes_kernel<2> : v <= 4 ? token_codes_kernel<4>
                                                                              : token_codes_kernel<8>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)M, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, x, (int)K, ldx, codes, scale);
}

}  // namespace ql
