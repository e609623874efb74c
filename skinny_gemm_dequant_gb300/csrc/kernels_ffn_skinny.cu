// Linear layers for few tokens that stream their weights once: y = x W^T on 4-bit integer weights
// with group scales, and the gated feed-forward block h = silu(a min(g, L)) clamp(u, -L, L),
// g = x Wg^T, u = x Wu^T, on 4-bit or bf16 weights.
//
//   w[n,k] = (q[n,k] - z[n,k/G]) * s[n,k/G],   q in 0..15, z in 0..127 (8 without zero points)
//   y[m,n] = bf16( sum_groups s * sum_{k in group} x[m,k] (q - z) )      (+ bias after the cast)
//
// q - z is exact in bf16 and a bf16 product is exact in fp32, so the warp MMA (bf16 operands,
// fp32 sums) adds exact products and each group's sum is multiplied by its scale once, in fp32:
// no weight is rounded.
//
// A CTA owns 16 or 32 weight rows (gated: 16 gate rows and the matching 16 up rows) and its
// eight warps split K; their sums meet in shared memory.  The weights are the MMA's A operand
// (16 rows), the tokens its N = 8 columns.  A lane loads whole 16-byte pieces of a row: which k
// an MMA slot stands for is free as long as both operands agree, so the pieces go to the MMA in
// the order in which they lie in memory.
#include <cuda_fp16.h>

#include "common.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "internal.h"

namespace ql {

namespace {

constexpr int kWarps = 8;

// nibble pairs of a word as bf16x2 of 128 + q: (e0,e4) (e1,e5) (e2,e6) (e3,e7); 0x4300 | q is the
// bf16 value 128 + q
__device__ __forceinline__ void nibbles_to_bf16(uint32_t w, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
}

// exact: both operands are integers of at most 8 significant bits
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float scale_to_f32(uint16_t bits, int fp16) {
  return fp16 ? __half2float(__ushort_as_half(bits)) : bf16_bits_to_f32(bits);
}

// lane t of four holds words 0..3 of 16-byte piece t; afterwards it holds word t of pieces 0..3
__device__ __forceinline__ void transpose4(uint4& v, int t) {
  uint32_t a[4] = {v.x, v.y, v.z, v.w};
  // exchange with lane t ^ 1: words of the other parity
#pragma unroll
  for (int p = 0; p < 4; p += 2) {
    const uint32_t give = (t & 1) ? a[p] : a[p + 1];
    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 1);
    if (t & 1)
      a[p] = got;
    else
      a[p + 1] = got;
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t give = (t & 2) ? a[p] : a[p + 2];
    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, 2);
    if (t & 2)
      a[p] = got;
    else
      a[p + 2] = got;
  }
  v = make_uint4(a[0], a[1], a[2], a[3]);
}

// One 64-byte block of every row per step: 128 k of 4-bit weights, 32 k of bf16 weights.
// MT: 16-row tiles per CTA; NT: 8-token tiles; FINE: groups shorter than 128 (4-bit only).
template <bool INT4, bool GATED, int MT, int NT, bool FINE>
__global__ void __launch_bounds__(kWarps * 32) ffn_skinny_kernel(const __grid_constant__ FfnSkinnyArgs a) {
  constexpr int KB = INT4 ? 128 : 32;
  __shared__ float red[kWarps][MT * 16][NT * 8 + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int m0 = blockIdx.y * (NT * 8);
  const int n0 = blockIdx.x * (GATED ? MT * 8 : MT * 16);

  // weight row of (tile, half) for this lane; rows past the end read the last row, unused
  int64_t row[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (GATED) {
        // even tiles are gate rows, odd tiles the up rows of the same outputs
        int n = n0 + (mt >> 1) * 16 + h * 8 + g;
        if (n >= a.N) n = a.N - 1;
        row[mt][h] = (mt & 1) ? (int64_t)a.N + n : n;
      } else {
        int n = n0 + mt * 16 + h * 8 + g;
        if (n >= a.N) n = a.N - 1;
        row[mt][h] = n;
      }
    }

  float acc[MT][NT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;

  const int nblk = (a.K + KB - 1) / KB;
  for (int b = warp; b < nblk; b += kWarps) {
    const int kl = b * KB + t * (KB / 4);  // first k of this lane's 16-byte piece
    uint4 wv[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        wv[mt][h] = kl < a.K ? ldg_stream(a.w + row[mt][h] * a.ldw_bytes + (int64_t)b * 64 + t * 16)
                             : make_uint4(0u, 0u, 0u, 0u);
    if constexpr (!INT4) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int m = m0 + nt * 8 + g;
        uint4 xv = make_uint4(0u, 0u, 0u, 0u);
        if (m < a.M && kl < a.K) xv = *reinterpret_cast<const uint4*>(a.x + (int64_t)m * a.ldx + kl);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma_bf16_16816(acc[mt][nt], wv[mt][0].x, wv[mt][1].x, wv[mt][0].y, wv[mt][1].y, xv.x, xv.y);
          mma_bf16_16816(acc[mt][nt], wv[mt][0].z, wv[mt][1].z, wv[mt][0].w, wv[mt][1].w, xv.z, xv.w);
        }
      }
    } else {
      // FINE: lane t takes word t of each 32-k piece, so that an MMA stays inside one group;
      // otherwise piece t whole (all four pieces share the group)
      if constexpr (FINE) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) transpose4(wv[mt][h], t);
      }
      uint32_t zero[MT][2];
      float sc[MT][2];
      float part[MT][NT][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kj = b * KB + (FINE ? 32 * j + 8 * t : 32 * t + 8 * j);
        if (j == 0 || FINE) {
          // the group's scale and zero point (FINE: of piece j)
          const int k0 = b * KB + (FINE ? 32 * j : 0);
          const int gi = k0 >> a.group_shift;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              sc[mt][h] = k0 < a.K ? scale_to_f32(a.scale[row[mt][h] * a.lds + gi], a.scale_fp16) : 0.f;
              const uint32_t z = (a.zero && k0 < a.K) ? a.zero[row[mt][h] * a.ldz + gi] : 8u;
              zero[mt][h] = (0x4300u | z) * 0x10001u;
            }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) part[mt][nt][i] = 0.f;
        }
        uint32_t bf[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int m = m0 + nt * 8 + g;
          uint4 xv = make_uint4(0u, 0u, 0u, 0u);
          if (m < a.M && kj < a.K) xv = *reinterpret_cast<const uint4*>(a.x + (int64_t)m * a.ldx + kj);
          bf[nt][0] = __byte_perm(xv.x, xv.z, 0x5410);
          bf[nt][1] = __byte_perm(xv.x, xv.z, 0x7632);
          bf[nt][2] = __byte_perm(xv.y, xv.w, 0x5410);
          bf[nt][3] = __byte_perm(xv.y, xv.w, 0x7632);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t q0[4], q1[4];
          const uint4 &v0 = wv[mt][0], &v1 = wv[mt][1];
          nibbles_to_bf16(j == 0 ? v0.x : j == 1 ? v0.y : j == 2 ? v0.z : v0.w, q0);
          nibbles_to_bf16(j == 0 ? v1.x : j == 1 ? v1.y : j == 2 ? v1.z : v1.w, q1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            q0[i] = sub_bf16x2(q0[i], zero[mt][0]);
            q1[i] = sub_bf16x2(q1[i], zero[mt][1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_bf16_16816(part[mt][nt], q0[0], q1[0], q0[1], q1[1], bf[nt][0], bf[nt][1]);
            mma_bf16_16816(part[mt][nt], q0[2], q1[2], q0[3], q1[3], bf[nt][2], bf[nt][3]);
          }
        }
        if (FINE || j == 3) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[mt][nt][i] = fmaf(sc[mt][i >> 1], part[mt][nt][i], acc[mt][nt][i]);
        }
      }
    }
  }

  // accumulator i of lane (g, t): row g + 8 (i >> 1), token 2t + (i & 1)
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][mt * 16 + g + 8 * (i >> 1)][nt * 8 + 2 * t + (i & 1)] = acc[mt][nt][i];
  __syncthreads();
  constexpr int OUT = GATED ? MT * 8 : MT * 16;
  for (int e = threadIdx.x; e < OUT * NT * 8; e += kWarps * 32) {
    const int o = e % OUT, m = m0 + e / OUT;
    const int n = n0 + o;
    if (n >= a.N || m >= a.M) continue;
    const int r = GATED ? (o >> 4) * 32 + (o & 15) : o;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += red[w][r][e / OUT];
    uint16_t yb;
    if constexpr (GATED) {
      float u = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) u += red[w][r + 16][e / OUT];
      yb = f32_to_bf16_rn(gated_act(v, u, a.alpha, a.limit));
    } else {
      yb = f32_to_bf16_rn(v);
      if (a.bias) yb = f32_to_bf16_rn(bf16_bits_to_f32(yb) + bf16_bits_to_f32(a.bias[n]));
    }
    a.y[(int64_t)m * a.ldy + n] = yb;
  }
}

template <bool INT4, bool GATED, int MT, int NT, bool FINE>
cudaError_t launch(const FfnSkinnyArgs& a, cudaStream_t st) {
  constexpr int OUT = GATED ? MT * 8 : MT * 16;
  const dim3 grid((unsigned)((a.N + OUT - 1) / OUT), (unsigned)((a.M + NT * 8 - 1) / (NT * 8)));
  ffn_skinny_kernel<INT4, GATED, MT, NT, FINE><<<grid, kWarps * 32, 0, st>>>(a);
  return cudaGetLastError();
}

template <bool INT4, bool GATED, bool FINE>
cudaError_t launch_nt(const FfnSkinnyArgs& a, cudaStream_t st) {
  if (a.M <= 8) return launch<INT4, GATED, 2, 1, FINE>(a, st);
  if (a.M <= 16) return launch<INT4, GATED, 2, 2, FINE>(a, st);
  return launch<INT4, GATED, 2, 4, FINE>(a, st);
}

}  // namespace

cudaError_t launch_ffn_skinny(bool int4, bool gated, const FfnSkinnyArgs& a, cudaStream_t st) {
  if (!int4) return launch_nt<false, true, false>(a, st);
  const bool fine = a.group_shift < 7;
  if (gated) return fine ? launch_nt<true, true, true>(a, st) : launch_nt<true, true, false>(a, st);
  return fine ? launch_nt<true, false, true>(a, st) : launch_nt<true, false, false>(a, st);
}

}  // namespace ql
