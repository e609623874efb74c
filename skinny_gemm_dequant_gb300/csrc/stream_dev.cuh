// Device helpers of the weight-streaming kernels (kernels_stream.cu, kernels_moe_few.cu): copies into a
// warp's ring, weights and activations to MMA operands.
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"
#include "stream.h"

namespace ql {

constexpr int kNone = 0x7FFFFFFF;  // the expert of a pair that is left out

struct Entry {  // one pass over an expert's weights
  uint16_t expert, first;
  int count;  // its pairs: s_pair[first, first + count)
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory; zeros, and no access to src, where `take` is false
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// all but the newest `left` copy groups have landed
__device__ __forceinline__ void cp_wait(int left) {
  switch (left) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
  }
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// bf16 patterns below 256 are linear (pattern p stands for p 2^-133), so a nibble in place is a
// number: one multiply-add gives (q - z) / 64, exactly
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t negz, uint32_t (&o)[4]) {
  const uint32_t v = w >> 8;
  o[0] = fma_bf16x2(w & 0x000F000Fu, 0x7F007F00u, negz);
  o[1] = fma_bf16x2(w & 0x00F000F0u, 0x7D007D00u, negz);
  o[2] = fma_bf16x2(v & 0x000F000Fu, 0x7F007F00u, negz);
  o[3] = fma_bf16x2(v & 0x00F000F0u, 0x7D007D00u, negz);
}
// eight activations in the order in which a word's codes come out: (0,4) (1,5) (2,6) (3,7)
__device__ __forceinline__ uint4 pair_up(uint4 x) {
  return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                    __byte_perm(x.y, x.w, 0x7632));
}
// 8-bit codes of a row of bf16 values whose largest magnitude is `top`: scale = top / 127, code =
// v / scale rounded half to even, both IEEE fp32 divisions.  Rounding v f, f = 127 / top, gives the same
// codes but for ties: with 8-bit mantissas v / top = a / (b 2^s), so v 127 / top is a tie only where b =
// 254, when all is exact, or v = top / 2, and it is never nearer than 1 / (510 2^s) to a tie otherwise
// (a = 254, b = 255: 126.50196), far more than what v f is off by, 2^-14 / 2^s.  Which way the quotient of
// top / 2 falls is asked once, and f moved to the side of 127 / top that falls the same way.
__device__ __forceinline__ float code_factor(float top) {
  if (top < 7.7037197775489436e-34f) return 0.f;  // 2^-110: zeros
  float f = __fdiv_rn(127.f, top);
  const float off = __fmaf_rn(f, top, -127.f);  // its sign is exact
  const bool down = __fdiv_rn(0.5f * top, __fdiv_rn(top, 127.f)) < 63.5f;
  if (down && off >= 0.f) f = __uint_as_float(__float_as_uint(f) - 1u);
  if (!down && off < 0.f) f = __uint_as_float(__float_as_uint(f) + 1u);
  return f;  // an infinite row: 0, which its infinities turn into NaN; a NaN stays
}
// two bf16 values as whole f16 numbers: v f + 1.5 2^23 is rounded once, to a whole number
__device__ __forceinline__ uint32_t quant2(uint32_t w, float f) {
  const float lo = fmaf(__uint_as_float(w << 16), f, 12582912.f) - 12582912.f;
  const float hi = fmaf(__uint_as_float(w & 0xFFFF0000u), f, 12582912.f) - 12582912.f;
  return pack_f16x2(lo, hi);
}
// the first MMA of a group's sum: no accumulator to clear
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Units of a CTA, of `total` that are cut into equal shares; `whole` units' sums meet before a result.  A
// share has a unit for each of the CTA's warps, which take them at once (fewer would only make more parts
// to join), and whole results where those are short.
__device__ __forceinline__ int unit_share(int total, int whole, int warps) {
  if (total == 0) return 1;
  int share = max((total + (int)gridDim.x - 1) / (int)gridDim.x, min(warps, whole));
  if (whole <= 2 * warps) share = (share + whole - 1) / whole * whole;
  return share;
}

// the parts c0..c1 of a DOWN tile, in the order of K: quad `at` (four rows of a token)
template <class Slot>
__device__ __forceinline__ float4 add_parts(Slot slot_of, int c0, int c1, int at) {
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int q = c0; q <= c1; ++q) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(slot_of(q, q == c0)) + at);
    y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
  }
  return y;
}
template <int R>
__device__ __forceinline__ void put4(const StreamArgs& p, int tile, int at, float4 y) {
  constexpr int Q = R / 4;
  const int row = tile * R + at % Q * 4;
  uint16_t* dst = reinterpret_cast<uint16_t*>(p.y) + (int64_t)(at / Q) * p.ldy + row;
  const float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (row + j < p.N) dst[j] = f32_to_bf16_rn(v[j]);
}

}  // namespace ql
