// The gated block's activation, its derivative, and the 8-bit form of a checkpoint.
#pragma once
#include <cstdint>

namespace ql {

// columns of a checkpoint row's halves (g, u): padded to whole groups of 128
__host__ __device__ __forceinline__ int64_t ckpt_pad(int64_t I) { return (I + 127) / 128 * 128; }

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// min(g, L) and clamp(u, -L, L) by comparisons, which let a NaN through
__device__ __forceinline__ float cap(float g, float limit) { return g > limit ? limit : g; }
__device__ __forceinline__ float clip(float u, float limit) { return u > limit ? limit : (u < -limit ? -limit : u); }

__device__ __forceinline__ float sigmoid_f32(float t) { return __fdividef(1.0f, 1.0f + __expf(-t)); }

// silu(a min(g, L)) * clamp(u, -L, L); the fast exponential and quotient are a few fp32 ulps off,
// far below the bf16 rounding of h.  Their quotient is 0 for denominators above 2^126, which
// sigmoid reaches only below t = -87, where t sigmoid(t) is under 2^-119.
__device__ __forceinline__ float gated_act(float g, float u, float alpha, float limit) {
  const float t = alpha * cap(g, limit);
  return t * sigmoid_f32(t) * clip(u, limit);
}

// dg = dh uc a silu'(t) [g <= L], du = dh silu(t) [|u| <= L], t = a min(g, L); a NaN in g or u
// stays one in the gradients that depend on it
__device__ __forceinline__ void gated_grad(float dh, float g, float u, float alpha, float limit, float& dg,
                                           float& du) {
  const float t = alpha * cap(g, limit);
  const float s = sigmoid_f32(t);
  du = (u > limit || u < -limit) ? 0.f : dh * t * s;
  dg = g > limit ? 0.f : dh * clip(u, limit) * alpha * (s + t * s * (1.0f - s));
}

// ------------------------------------------------------------------ 8-bit checkpoint
// scale = amax / 127, codes rint(v * (127 / amax)): one division a group, and the product is within
// 2^-16 of v / scale, so that only a value that near to a tie gets the other of its two codes.  Groups whose amax is under 2^-100 are kept as
// zeros (127 / amax would overflow); an infinity or a NaN makes the scale a NaN, so that every value
// of the group reads back as one.
__device__ __forceinline__ float ckpt_scale(float amax, float& inv) {
  if (amax < 0x1p-100f) {
    inv = 0.f;
    return 0.f;
  }
  inv = 127.0f / amax;
  return amax / 127.0f + (amax - amax);
}
// 32 codes.  Added to 1.5 2^23 a value is rounded to the nearest whole number, ties to even, which
// then stands in the sum's low bits: |v| inv <= 127 (1 + 2^-23).  A conversion per code goes through
// the pipe of the exponentials, four lanes a cycle (333 x 2040 x 1024: this epilogue 5.3 us, so 4.8)
__device__ __forceinline__ void ckpt_codes32(const float* v, float inv, uint32_t* w) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t c[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) c[b] = __float_as_uint(fmaf(v[4 * j + b], inv, 0x1.8p23f));
    w[j] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  }
}
__device__ __forceinline__ void ckpt_values8(uint2 c, float scale, float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)(int8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3))) * scale;
}
__device__ __forceinline__ void bf16_values8(uint4 c, float* v) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __uint_as_float((j & 1) ? (w[j >> 1] & 0xFFFF0000u) : (w[j >> 1] << 16));
}

}  // namespace ql
