// The two launches of a mixture-of-experts layer for up to 64 tokens (bf16, 8-bit and 4-bit weights).
//
//   GATE_UP  g = W13[e][0:I] x_m, u = W13[e][I:2I] x_m for every routed pair (m, j) with expert e,
//            h = bf16( silu(a min(g, L)) clamp(u, -L, L) )
//   DOWN     y_m = bf16( sum_j w_(m,j) W2[e] h_(m,j) )
//
// 8-bit weights: tokens (GATE_UP) and h (DOWN) are quantised here, scale = max|v| / 127 over the
// row, code = v / scale rounded half to even; products of codes are exact in fp32, sums of
// 1024 k too.  4-bit weights: q - z is exact in bf16, a group's fp32 sum is multiplied by its scale once.
// h is rounded to bf16 once (the products' operand).  GATE_UP's 8-bit sums are whole numbers; all others are
// fp32, in DOWN of 8-bit weights over runs of at most 1024 k whose own sums are exact.
//
// Both kernels are persistent, one CTA per SM, and stream a chosen expert's weights once for 8 of its
// tokens through rings of the warps' own (cp.async: no warp waits for another), the weights as the warp
// MMA's A operand and tokens as its columns.  At these counts of tokens the tensor cores idle either way
// and what counts is the bytes in flight.
// GATE_UP: all tokens stay in shared memory as MMA operands (where they do not fit, the launch of
// kernels_stream.cu takes over: gate_up_few_takes); a warp takes 8 gate rows and the 8 up rows of the same
// outputs over the whole K, so that nothing is joined and h is made in its registers.  K cut over
// warps and joined through shared memory took 40 us where this took 35 in both launches (4-bit, one
// token, 8 experts of 2048x4096), 55 and 46 with 8-bit weights.
// DOWN: the units (32 rows by 64 or 128 k) of a tile are all its experts' K in a row; they are cut evenly
// over the warps of all CTAs.  A warp adds an expert's products into registers and, where the expert
// changes, w_(m,j) times them into its results of the tile, [tokens][32] in shared memory.  64-row tiles
// leave fewer warps room beside 64 tokens' results: bf16 1801 and 1685 us, 4-bit 806 and 787 us (8 of
// 256 experts), 78 and 105 us (bf16, 16 experts of 1032x2056); up to 16 tokens they are even.
// GATE_UP hands DOWN the routing, so that it is worked out once (39 to 36 us with one token).
// 4-bit weights become (q - z) / 64 by a multiply-add a pair.  Raw nibbles as bf16 numbers q 2^-133, x times 2^64
// and the zero point taken out by sums of x a group save those, but x of 2^63 and more overflows and the sum
// is off relative to (q + z) |x|; measured: 35.0 and 35.9 us (one token, groups of 128 without zero points),
// 38.8 and 37.5 with them, 68.0 and 65.8 in groups of 32, 98 and 94 (13 tokens, 60 experts of 1376x2080).
//
// Measured, both launches of 8 experts of 2048x4096 a token on one of 256 (bytes: chosen experts'
// weights): bf16 one token 70 us (5.7 TB/s), 24 tokens 982 us (7.0 TB/s); 8-bit one token 46 us
// (4.4 TB/s), 16 tokens 410 us (6.3 TB/s); 4-bit one token 36 us (2.9 TB/s), 12 tokens 208 us
// (5.1 TB/s).  Many tokens are bound by HBM.  One token: 10 of the microseconds are two launches' starts,
// routing, the tokens' way into shared memory and the joining of tiles.  4-bit weights are bound by latency
// beside that: four warps a scheduler, each alone in its chain of loads, nibbles, scales by shuffles and
// products, issue 1.3 to 1.6 instructions a cycle an SM with DRAM at 12 to 39 % and the tensor pipe at 6 to 18 %
// (groups below 128 take twice the scale work).  An expert's tokens beyond 8 read its weights again, in DOWN nearly
// always from HBM: the rows that all warps go through between two passes are larger than L2.
#include <algorithm>

#include "common.cuh"
#include "ffn_act.cuh"
#include "moe_dispatch.cuh"
#include "stream.h"
#include "stream_dev.cuh"

namespace ql {

namespace {

constexpr int kGuWarps = 16;
constexpr int kDnRows = 32, kDnFew = 20;  // DOWN: rows of a tile; tokens that leave 4-bit weights 16 warps
constexpr int kSmem = 226 * 1024;
constexpr int kStage = 16 * 128, kGuDepth = 4;  // GATE_UP's rings: bytes of a stage, stages at most
// shared memory of GATE_UP for lists; the tokens have the rest
__host__ __device__ constexpr int gu_list_bytes(int pairs) {
  return (pairs * 16 + kMoeMaxTokens * 4 + 127) & ~127;  // entries, ids, sorted pairs and tokens; scales
}

// k of a stage
__host__ __device__ constexpr int gu_k(int fmt) { return fmt == STREAM_INT4 ? 256 : fmt == STREAM_INT8 ? 128 : 64; }

// slot of 16-byte piece c of row m of MMA operands of BYTES a row, for the reads below
template <int FMT, bool FINE>
__device__ __forceinline__ int xslot(int c, int m) {
  if (FMT == STREAM_BF16) return c ^ ((m & 1) << 2);
  if (FMT == STREAM_INT8) return c ^ (m & 1);
  return c ^ (FINE ? (m & 1) << 2 : (c >> 3) + ((m & 1) << 1));
}
__device__ __forceinline__ int wslot(int c, int r) { return c ^ (((r & 1) << 2) | ((r >> 1) & 3)); }

// ------------------------------------------------------------------ GATE_UP
// DEPTH: stages of a ring, or 0: as the argument says
template <int FMT, int DEPTH, bool FINE, bool ZP>
__global__ void __launch_bounds__(kGuWarps * 32, 1)
    gate_up_kernel(const __grid_constant__ StreamArgs p, int x_bytes, int lists, int depth_arg) {
  constexpr bool I8 = FMT == STREAM_INT8, I4 = FMT == STREAM_INT4;
  constexpr int KS = gu_k(FMT), XB = FMT == STREAM_BF16 ? 128 : 256;  // k of a stage; bytes of a token's x block
  constexpr int XK = FMT == STREAM_BF16 ? 64 : 128, SB = KS / XK;     // k of an x block; blocks of a stage
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int P = p.M * p.topk;
  const int nstage = (p.K + KS - 1) / KS, nxb = nstage * SB;  // x is zero past K

  // shared memory: x blocks [nxb][M], lists, rings
  uint8_t* ring_base = smem + x_bytes + lists;
  Lists l;
  l.entries = reinterpret_cast<Entry*>(smem + x_bytes);
  l.ids = reinterpret_cast<int*>(l.entries + P);
  float* s_xs = reinterpret_cast<float*>(l.ids + P);
  l.pair = reinterpret_cast<uint16_t*>(s_xs + kMoeMaxTokens);
  l.tok = l.pair + P;
  l.keys = reinterpret_cast<int*>(ring_base);  // the rings are filled later
  l.heads = reinterpret_cast<Entry*>(l.keys + (P + 3) / 4 * 4);
  __shared__ unsigned s_top[kMoeMaxTokens];
  __shared__ float s_inv[kMoeMaxTokens];
  __shared__ int s_one, s_next;

  if (I8 && threadIdx.x < kMoeMaxTokens) s_top[threadIdx.x] = 0u;
  if (threadIdx.x == 0) s_next = 0;
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();

  // the first warps route, the others take x meanwhile
  const int routing = p.M <= kGuWarps ? min(p.M, kGuWarps / 2) : kGuWarps, vecs = nxb * (XK / 8);
  const int chunks = (vecs * p.M + 63) / 64;
  auto stage_x = [&]() {
    // a warp takes the next 64 pieces, so that those that route join in later; pieces of a token are
    // neighbours, 16 lanes hold a block of 128 k
#pragma unroll 1
    for (;;) {
      int next = 0;
      if (lane == 0) next = atomicAdd(&s_next, 1);
      next = __shfl_sync(0xffffffffu, next, 0);
      if (next >= chunks) break;
      uint4 x2[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int i = next * 64 + q * 32 + lane, m = i / vecs, v = i - m * vecs;
        x2[q] = make_uint4(0u, 0u, 0u, 0u);
        if (m < p.M && v * 8 < p.K) x2[q] = *reinterpret_cast<const uint4*>(p.x + m * p.ldx + v * 16);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int i = next * 64 + q * 32 + lane;
        const bool on = i < vecs * p.M;
        const int m = on ? i / vecs : 0, v = i - m * vecs, b = v / (XK / 8), c = v % (XK / 8);
        uint4 x = x2[q];
        if constexpr (I8) {
          const float inv = s_inv[m];
          x = make_uint4(quant2(x.x, inv), quant2(x.y, inv), quant2(x.z, inv), quant2(x.w, inv));
        }
        if constexpr (I4) x = pair_up(x);
        if (on) *reinterpret_cast<uint4*>(smem + (size_t)(b * p.M + m) * XB + xslot<FMT, FINE>(c, m) * 16) = x;
      }
    }
  };
  auto top_x = [&](int first, int warps) {
    // a warp takes a token, or where they are few a segment of one
    const int segments = max(1, warps / p.M), vecs_row = p.K / 8;
#pragma unroll 1
    for (int i = first; i < p.M * segments; i += warps) {
      const int m = i / segments, s = i - m * segments;
      float top = 0.f;
#pragma unroll 4
      for (int v = vecs_row * s / segments + lane; v < vecs_row * (s + 1) / segments; v += 32) {
        const uint4 x = *reinterpret_cast<const uint4*>(p.x + m * p.ldx + v * 16);
        const uint32_t q[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          top = max_nan(max_nan(top, fabsf(__uint_as_float(q[j] << 16))), fabsf(__uint_as_float(q[j] & 0xFFFF0000u)));
      }
      // as whole numbers: a NaN is above all
      const unsigned most = __reduce_max_sync(0xffffffffu, __float_as_uint(top) & 0x7FFFFFFFu);
      if (lane == 0) atomicMax(&s_top[m], most);
    }
  };
  int ne, most = 1;
  if (warp < routing) {
    if (p.M == 1)
      s_one = route_one(p, l);
    else
      route(p, l, routing);
  }
  if constexpr (I8) {
    if (routing == kGuWarps)
      top_x(warp, kGuWarps);
    else if (warp >= routing)
      top_x(warp - routing, kGuWarps - routing);
  }
  if constexpr (!I8) stage_x();
  __syncthreads();
  if constexpr (I8) {
    if (threadIdx.x < p.M) {
      const float top = __uint_as_float(s_top[threadIdx.x]);
      s_xs[threadIdx.x] = __fdiv_rn(top, 127.f);
      s_inv[threadIdx.x] = code_factor(top);
    }
    __syncthreads();
  }
  ne = p.M == 1 ? s_one : dispatch<kGuWarps>(p, l, kPerEntry, most);

  const int depth = DEPTH > 0 ? DEPTH : depth_arg;
  const int otiles = p.N / 8, total = ne * otiles;
  const int step = (int)gridDim.x * kGuWarps;
  const uint32_t ring = smem_addr(ring_base) + (uint32_t)(warp * depth * kStage);

  // a lane copies 16-byte piece cc of rows cr and cr + 4, gate and up
  const int cr = lane >> 3, cc = lane & 7;
  const uint32_t dst0 = (uint32_t)(cr * 128 + wslot(cc, cr) * 16), dst1 = (uint32_t)((cr + 4) * 128 + wslot(cc, cr + 4) * 16);
  const int64_t up = (int64_t)p.N * p.ldw, four = 4 * p.ldw;
  const int kbytes = I4 ? p.K / 2 : I8 ? p.K : p.K * 2;
  int f_tile = (int)blockIdx.x + warp * (int)gridDim.x, f_left = 0;  // bytes of a row to copy
  const uint8_t *f_gate = nullptr, *f_up = nullptr;
  auto fetch = [&](uint32_t at) {
    if (f_left <= 0 && f_tile < total) {
      const int a = f_tile / otiles, o = f_tile - a * otiles;
      f_gate = p.w + l.entries[a].expert * p.w_estride + (int64_t)(o * 8 + cr) * p.ldw + cc * 16;
      f_up = f_gate + up;
      f_left = kbytes;
      f_tile += step;
    }
    if (f_left > 0) {
      const bool in = cc * 16 < f_left;
      cp16(at + dst0, f_gate, in);
      cp16(at + dst1, f_gate + four, in);
      cp16(at + 1024 + dst0, f_up, in);
      cp16(at + 1024 + dst1, f_up + four, in);
      f_gate += 128;
      f_up += 128;
      f_left -= 128;
    }
    cp_commit();
  };
#pragma unroll 1
  for (int d = 0; d < depth - 1; ++d) fetch(ring + d * kStage);

  if constexpr (I8) {  // (the weights are on their way)
    stage_x();
    __syncthreads();
  }
  // for the next launch, by the warps that have the fewest tiles
  if (blockIdx.x == gridDim.x - 1 && warp == kGuWarps - 2) hand_lists(p, l, ne, most);
  if (gridDim.x - 1 - blockIdx.x < p.M && warp == kGuWarps - 1) hand_weights(p, l, gridDim.x - 1 - blockIdx.x);

  const uint32_t end = (uint32_t)(depth * kStage);
  uint32_t slot = 0;  // byte offset of the stage in the ring
  const uint32_t w0_at = ring + (uint32_t)(g * 128 + wslot(t, g) * 16), w1_at = w0_at ^ 64u;  // pieces t, 4 + t
#pragma unroll 1
  for (int tile = (int)blockIdx.x + warp * (int)gridDim.x; tile < total; tile += step) {
    const int a = tile / otiles, o = tile - a * otiles;
    const Entry en = l.entries[a];
    const int xg = l.tok[en.first + min(g, en.count - 1)];  // the token of this lane's B column
    uint32_t xb = smem_addr(smem) + (uint32_t)(xg * XB);  // its row of the x block
    // scales: 4-bit: lane (g, t) those of gate (t < 2) or up row g, of block t % 2 of a stage
    constexpr int NS = FINE ? 4 : 1;
    uint16_t s_next[NS];
    uint8_t z_next[NS];
    const uint16_t* sp = nullptr;
    const uint8_t* zp = nullptr;
    float ws[2] = {1.f, 1.f};
    auto scales = [&](int s) {
      if constexpr (I4) {
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const int k = s * KS + (t & 1) * 128 + j * 32;
          const int gi = min(k, p.K - 1) >> p.group_shift;
          s_next[j] = k < p.K ? sp[gi] : (uint16_t)0;  // past the end: sums of zeros
          if (ZP) z_next[j] = zp[gi];
        }
      }
    };
    {
      const int64_t row = o * 8 + g + (I4 && t >= 2 ? (int64_t)p.N : 0);
      if constexpr (I4) {
        sp = reinterpret_cast<const uint16_t*>(p.scale) + en.expert * p.s_estride + row * p.lds;
        if (ZP) zp = p.zero + en.expert * p.z_estride + row * p.ldz;
        scales(0);
      }
      if constexpr (I8) {
        const float* s = reinterpret_cast<const float*>(p.scale) + en.expert * p.s_estride + row;
        ws[0] = s[0];
        ws[1] = s[p.N];
      }
    }
    // token columns 2t, 2t + 1 of the sums
    const int c0 = l.tok[en.first + min(2 * t, en.count - 1)], c1 = l.tok[en.first + min(2 * t + 1, en.count - 1)];
    float acc[4] = {};
    int whole[4] = {};
#pragma unroll 1
    for (int s = 0; s < nstage; ++s) {
      cp_wait(depth - 2);
      __syncwarp();  // every lane's copies of this stage have landed, and the stage before is read
      fetch(ring + (slot == 0 ? end : slot) - kStage);
      const uint32_t wa[2] = {w0_at + slot, w1_at + slot};
      const uint32_t wf = ring + slot + g * 128 + t * 4, wx = wslot(0, g) * 16;  // FINE: word t of piece c at c * 16 ^ wx
      slot = slot + kStage == end ? 0u : slot + kStage;
      float sc[NS];  // scale and zero point (as bf16x2 of -z / 64) of this lane's row and block
      uint32_t nz[NS];
      if constexpr (I4) {
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          sc[j] = p.scale_fp16 ? __half2float(__ushort_as_half(s_next[j])) : bf16_bits_to_f32(s_next[j]);
          // z's pattern stands for z 2^-133, times -2^127
          if (ZP) nz[j] = fma_bf16x2(z_next[j] * 0x10001u, 0xFF00FF00u, 0u);
        }
        if (s + 1 < nstage) scales(s + 1);
      }
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) {
        if constexpr (I4) {
          uint32_t wv[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (FINE) {
              // word t of every 32-k piece, so that an MMA stays inside one group
#pragma unroll
              for (int j = 0; j < 4; ++j) wv[h][j] = lds4(wf + h * 1024 + ((4 * sb + j) * 16 ^ wx));
            } else {
              const uint4 v = lds16(wa[sb] + h * 1024);
              wv[h][0] = v.x;
              wv[h][1] = v.y;
              wv[h][2] = v.z;
              wv[h][3] = v.w;
            }
          }
          float grp[4], f[2];
          uint32_t negz[2];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 bx = lds16(xb + xslot<FMT, FINE>(FINE ? 4 * j + t : 4 * t + j, xg) * 16);
            if (j == 0 || FINE) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                f[h] = __shfl_sync(0xffffffffu, sc[FINE ? j : 0], g * 4 + h * 2 + sb);
                negz[h] = ZP ? __shfl_sync(0xffffffffu, nz[FINE ? j : 0], g * 4 + h * 2 + sb) : 0xBE00BE00u;
              }
            }
            uint32_t q0[4], q1[4];
            codes_to_bf16(wv[0][j], negz[0], q0);
            codes_to_bf16(wv[1][j], negz[1], q1);
            if (j == 0 || FINE)
              mma_first(grp, q0[0], q1[0], q0[1], q1[1], bx.x, bx.y);
            else
              mma_bf16_16816(grp, q0[0], q1[0], q0[1], q1[1], bx.x, bx.y);
            mma_bf16_16816(grp, q0[2], q1[2], q0[3], q1[3], bx.z, bx.w);
            if (FINE || j == 3) {
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[i] = fmaf(f[i >> 1], grp[i], acc[i]);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 w0 = lds16(wa[j]), w1 = lds16(wa[j] + 1024);
            if constexpr (I8) {
              const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, hi[4] = {w1.x, w1.y, w1.z, w1.w};
              const uint4 xa = lds16(xb + xslot<FMT, FINE>(8 * j + 2 * t, xg) * 16);
              const uint4 xc = lds16(xb + xslot<FMT, FINE>(8 * j + 2 * t + 1, xg) * 16);
              const uint32_t b[8] = {xa.x, xa.y, xa.z, xa.w, xc.x, xc.y, xc.z, xc.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t a0, a1, a2, a3;
                s8x4_to_f16x2x2(lo[i], a0, a2);
                s8x4_to_f16x2x2(hi[i], a1, a3);
                mma_f16_16816(acc, a0, a1, a2, a3, b[2 * i], b[2 * i + 1]);
              }
            } else {
              const uint4 x = lds16(xb + xslot<FMT, FINE>(4 * j + t, xg) * 16);
              mma_bf16_16816(acc, w0.x, w1.x, w0.y, w1.y, x.x, x.y);
              mma_bf16_16816(acc, w0.z, w1.z, w0.w, w1.w, x.z, x.w);
            }
          }
        }
        xb += (uint32_t)(p.M * XB);
      }
      if (I8 && ((s & 7) == 7 || s == nstage - 1)) {  // 1024 k: sums of at most 2^24
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          whole[i] += __float2int_rn(acc[i]);
          acc[i] = 0.f;
        }
      }
    }
    // a lane holds gate (0, 1) and up (2, 3) of output g for columns 2t, 2t + 1
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = 2 * t + i < en.count;
      float gv = acc[i], uv = acc[2 + i];
      if constexpr (I8) {
        const float xs = s_xs[i ? c1 : c0];
        gv = (float)whole[i] * xs * ws[0];
        uv = (float)whole[2 + i] * xs * ws[1];
      }
      if constexpr (I4) {
        gv *= 64.f;
        uv *= 64.f;
      }
      const uint16_t hb = f32_to_bf16_rn(gated_act(gv, uv, p.alpha, p.limit));
      const int pair = l.pair[en.first + min(2 * t + i, en.count - 1)];
      if (in) p.h[pair * p.ldh + o * 8 + g] = hb;
      if constexpr (I8) {
        unsigned top = (unsigned)(hb & 0x7FFF) << 16;
#pragma unroll
        for (int q = 4; q < 32; q <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, q));
        if (in && g == 0) atomicMax(p.amax + pair, top);
      }
    }
  }
}

// ------------------------------------------------------------------ DOWN
// W: warps
template <int FMT, int W, bool FINE, bool ZP>
__global__ void __launch_bounds__(W * 32, 1) down_kernel(const __grid_constant__ StreamArgs p, int lists) {
  constexpr bool I8 = FMT == STREAM_INT8, I4 = FMT == STREAM_INT4;
  constexpr int R = kDnRows, THREADS = W * 32, MT = R / 16, kPitch = R + 4;
  constexpr int KU = FMT == STREAM_BF16 ? 64 : 128, WB = I4 ? 64 : 128, XB = FMT == STREAM_BF16 ? 128 : 256;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int P = p.M * p.topk, ysize = p.M * kPitch;

  // shared memory: the warps' results of the tile they are in [W][M][kPitch], lists, rings
  float* s_y = reinterpret_cast<float*>(smem);
  Entry* entries = reinterpret_cast<Entry*>(s_y + W * ysize);
  float* s_wt = reinterpret_cast<float*>(entries + P);  // by pair; 8-bit: times the scale of h
  float* s_inv = s_wt + P;
  uint16_t* s_pair = reinterpret_cast<uint16_t*>(s_inv + P);
  uint16_t* s_tok = s_pair + P;
  uint8_t* rings = smem + lists;
  __shared__ int s_last[3];

  float* y = s_y + warp * ysize;
  for (int i = lane; i < ysize; i += 32) y[i] = 0.f;
  pdl_wait();
  pdl_launch_dependents();
  const Handed& from_gu = *reinterpret_cast<const Handed*>(p.handed);
  const int ne = from_gu.entries, xt = from_gu.most;
#pragma unroll 1
  for (int i = threadIdx.x; i < P; i += THREADS) {
    if (i < ne) entries[i] = from_gu.entry[i];
    s_pair[i] = from_gu.pair[i];
    s_tok[i] = from_gu.tok[i];
    float wt = from_gu.weight[i];
    if constexpr (I8) {
      const float top = __uint_as_float(p.amax[i]);
      wt *= __fdiv_rn(top, 127.f);
      s_inv[i] = code_factor(top);
    }
    s_wt[i] = wt;
  }
  __syncthreads();

  const int nblk = (p.K + KU - 1) / KU, tiles = (p.N + R - 1) / R, whole = ne * nblk, total = tiles * whole;
  if (total == 0) {  // nothing was dispatched
    for (int i = blockIdx.x * THREADS + threadIdx.x; i < p.M * p.N; i += gridDim.x * THREADS)
      reinterpret_cast<uint16_t*>(p.y)[(int64_t)(i / p.N) * p.ldy + i % p.N] = 0;
    return;
  }
  const int share = unit_share(total, whole, W);
  const int u0 = min(total, (int)blockIdx.x * share), u1 = min(total, u0 + share);
  auto bound = [&](int w) { return u0 + (u1 - u0) * w / W; };  // (at most 2^26 units a CTA)
  const int v0 = bound(warp), v1 = bound(warp + 1);
  const int stage = R * WB + xt * XB, depth = min(6, (kSmem - lists) / (W * stage));
  const uint32_t ring = smem_addr(rings) + (uint32_t)(warp * depth * stage);

  constexpr int LPR = WB / 16, RPI = 32 / LPR;  // lanes per weight row, rows per copy
  constexpr int LPT = XB / 16, TPI = 32 / LPT;  // lanes per token row, tokens per copy
  const int cr = lane / LPR, cc = lane % LPR, tr = lane / LPT, tc = lane % LPT;
  auto swz = [](int c, int r) { return c ^ ((((r & 1) << 2) | ((r >> 1) & 3)) & (LPR - 1)); };
  const uint32_t w_dst = (uint32_t)(cr * WB + swz(cc, cr) * 16);

  struct At {  // a unit: its number, block of K, entry, tile
    int u, kb, a, tile;
  };
  auto set = [&](int u) {
    At w;
    w.u = u;
    w.tile = u / whole;
    const int r = u - w.tile * whole;
    w.a = r / nblk;
    w.kb = r - w.a * nblk;
    return w;
  };
  auto next = [&](At& w) {
    ++w.u;
    if (++w.kb == nblk) {
      w.kb = 0;
      if (++w.a == ne) {
        w.a = 0;
        ++w.tile;
      }
    }
  };

  At f = set(v0);
  int f_valid = 0, f_toks = 0, f_first = 0;
  const uint8_t* f_w = nullptr;
  const int64_t wstep = (int64_t)RPI * p.ldw;
  auto target = [&]() {
    const Entry en = entries[f.a];
    f_valid = p.N - f.tile * R - cr;
    f_toks = en.count;
    f_first = en.first;
    f_w = p.w + en.expert * p.w_estride + (int64_t)(f.tile * R + cr) * p.ldw + cc * 16;
  };
  auto fetch = [&](uint32_t at) {
    const int kx = f.kb * XB + tc * 16;
#pragma unroll 1
    for (int m = tr; m < f_toks; m += TPI)
      cp16(at + R * WB + m * XB + xslot<FMT, FINE>(tc, m) * 16, p.x + s_pair[f_first + m] * p.ldx + kx, kx < p.K * 2);
    const int k = f.kb * WB + cc * 16;
    const int valid = k < (I4 ? p.K / 2 : I8 ? p.K : p.K * 2) ? f_valid : -R;
    const uint8_t* src = f_w + (int64_t)f.kb * WB;
#pragma unroll
    for (int i = 0; i < R / RPI; ++i) {
      // (rows 4 apart: the slot differs in bit 1)
      cp16((at + w_dst + i * RPI * WB) ^ (RPI == 4 && (i & 1) ? 32u : 0u), src, i * RPI < valid);
      src += wstep;
    }
  };

  // scales of a unit (4-bit) or of an entry (8-bit): a lane reads those of row `lane` of the tile
  static_assert(R == 32, "a row for each lane");
  constexpr int NS = FINE ? 4 : 1;
  uint16_t s_next[NS];  // as loaded: turning them into numbers here would wait for them
  uint8_t z_next[NS];
  const uint16_t* sp = nullptr;
  const uint8_t* zp = nullptr;
  auto scale_rows = [&](const At& w) {
    if constexpr (I4) {
      const int e = entries[w.a].expert;
      const int64_t n = min(w.tile * R + lane, p.N - 1);
      sp = reinterpret_cast<const uint16_t*>(p.scale) + e * p.s_estride + n * p.lds;
      if (ZP) zp = p.zero + e * p.z_estride + n * p.ldz;
    }
  };
  auto scales = [&](int kb) {
    if constexpr (I4) {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const int k = kb * KU + j * 32;
        const int gi = min(k, p.K - 1) >> p.group_shift;
        s_next[j] = k < p.K ? sp[gi] : (uint16_t)0;  // past the end: sums of zeros
        if (ZP) z_next[j] = zp[gi];
      }
    }
  };

  float part[MT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) part[mt][i] = 0.f;

  const int pre = depth - 1;
#pragma unroll 1
  for (int d = 0; d < pre; ++d) {
    if (f.u < v1) {
      if (d == 0 || f.kb == 0) target();
      fetch(ring + d * stage);
    }
    cp_commit();
    next(f);
  }

  At c = set(v0);
  int first_u = v0;  // of the tile's units that this warp has added
  uint32_t slot = 0, to_slot = pre;
  int count = 0, row = 0, first = 0;  // the entry's pairs; this lane's B column among them
  float inv = 0.f;
  float ws = 0.f;
  auto enter = [&]() {
    const Entry en = entries[c.a];
    count = en.count;
    first = en.first;
    row = min(g, count - 1);
    if constexpr (I8) {
      inv = s_inv[s_pair[first + row]];
      const int n = c.tile * R + lane;
      ws = n < p.N ? reinterpret_cast<const float*>(p.scale)[en.expert * p.s_estride + n] : 0.f;
    }
  };
  // an entry's sums, times the tokens' weights, into the tile's results: a lane has its own rows of columns
  // 2t and 2t + 1, whose tokens differ
  auto fold = [&]() {
    float sc[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        sc[mt][h] = I8 ? __shfl_sync(0xffffffffu, ws, mt * 16 + h * 8 + g) : I4 ? 64.f : 1.f;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      if (2 * t + q < count) {
        const int at = first + 2 * t + q;
        const float wt = s_wt[s_pair[at]];
        float* to = y + s_tok[at] * kPitch + g;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float& v = to[mt * 16 + 8 * h];
            v = fmaf(wt, sc[mt][h] * part[mt][2 * h + q], v);
          }
      }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[mt][i] = 0.f;
  };
  auto put = [&](int tile, int i, float v) {  // element i of [M][R]
    const int n = tile * R + i % R;
    if (n < p.N) reinterpret_cast<uint16_t*>(p.y)[(int64_t)(i / R) * p.ldy + n] = f32_to_bf16_rn(v);
  };
  // results of the tile that a warp begins in, where it goes on to another one: [CTA][W][M][R]
  auto head_of = [&](int w) { return p.heads + ((int64_t)blockIdx.x * W + w) * (p.M * R); };
  // the end of this warp's part [first_u, end) of a tile, which is not its last: written, or left
  auto finish = [&](int tile) {
    const bool all = first_u == tile * whole;
    __syncwarp();
    for (int i = lane; i < p.M * R; i += 32) {
      float& v = y[i / R * kPitch + i % R];
      if (all)
        put(tile, i, v);
      else
        __stcg(head_of(warp) + i, v);
      v = 0.f;
    }
    __syncwarp();
  };

  int folded = 0;
  if (c.u < v1) {
    enter();
    scale_rows(c);
    scales(c.kb);
  }
#pragma unroll 1
  while (c.u < v1) {
    cp_wait(pre - 1);
    __syncwarp();  // every lane's copies of this unit have landed, and the unit before is read
    if (f.u < v1) {
      if (f.kb == 0) target();
      fetch(ring + to_slot * stage);
    }
    cp_commit();
    next(f);
    if (++to_slot == (uint32_t)depth) to_slot = 0;
    const uint32_t wat = ring + slot * stage + g * WB, xat = ring + slot * stage + R * WB + row * XB;
    if (++slot == (uint32_t)depth) slot = 0;
    float scl[NS];  // scale and zero point (as bf16x2 of -z / 64) of this lane's rows
    uint32_t nzl[NS];
    At n = c;
    next(n);
    if constexpr (I4) {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        scl[j] = p.scale_fp16 ? __half2float(__ushort_as_half(s_next[j])) : bf16_bits_to_f32(s_next[j]);
        // z's pattern stands for z 2^-133, times -2^127
        if (ZP) nzl[j] = fma_bf16x2(z_next[j] * 0x10001u, 0xFF00FF00u, 0u);
      }
      if (n.u < v1) {
        if (n.kb == 0) scale_rows(n);
        scales(n.kb);
      }
    }

    if constexpr (I4) {
      uint4 bx[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) bx[j] = pair_up(lds16(xat + xslot<FMT, FINE>(FINE ? j * 4 + t : t * 4 + j, row) * 16));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        // rows g, g + 8 of the row tile
        uint32_t wv[2][4], negz[2];
        float sc[2], grp[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t at = wat + (mt * 16 + h * 8) * WB;
          if constexpr (FINE) {
            // word t of every 32-k piece, so that an MMA stays inside one group
#pragma unroll
            for (int j = 0; j < 4; ++j) wv[h][j] = lds4(at + swz(j, g) * 16 + t * 4);
          } else {
            const uint4 v = lds16(at + swz(t, g) * 16);
            wv[h][0] = v.x;
            wv[h][1] = v.y;
            wv[h][2] = v.z;
            wv[h][3] = v.w;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j == 0 || FINE) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              sc[h] = __shfl_sync(0xffffffffu, scl[FINE ? j : 0], mt * 16 + h * 8 + g);
              negz[h] = ZP ? __shfl_sync(0xffffffffu, nzl[FINE ? j : 0], mt * 16 + h * 8 + g) : 0xBE00BE00u;
            }
          }
          uint32_t q0[4], q1[4];
          codes_to_bf16(wv[0][j], negz[0], q0);
          codes_to_bf16(wv[1][j], negz[1], q1);
          if (j == 0 || FINE)
            mma_first(grp, q0[0], q1[0], q0[1], q1[1], bx[j].x, bx[j].y);
          else
            mma_bf16_16816(grp, q0[0], q1[0], q0[1], q1[1], bx[j].x, bx[j].y);
          mma_bf16_16816(grp, q0[2], q1[2], q0[3], q1[3], bx[j].z, bx[j].w);
          if (FINE || j == 3) {
#pragma unroll
            for (int i = 0; i < 4; ++i) part[mt][i] = fmaf(sc[i >> 1], grp[i], part[mt][i]);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t b[8];
        if constexpr (I8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 v = lds16(xat + xslot<FMT, FINE>(8 * j + 2 * t + i, row) * 16);
            b[4 * i] = quant2(v.x, inv);
            b[4 * i + 1] = quant2(v.y, inv);
            b[4 * i + 2] = quant2(v.z, inv);
            b[4 * i + 3] = quant2(v.w, inv);
          }
        } else {
          const uint4 v = lds16(xat + xslot<FMT, FINE>(4 * j + t, row) * 16);
          b[0] = v.x;
          b[1] = v.y;
          b[2] = v.z;
          b[3] = v.w;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint4 w0 = lds16(wat + (mt * 16) * WB + swz(4 * j + t, g) * 16);
          const uint4 w1 = lds16(wat + (mt * 16 + 8) * WB + swz(4 * j + t, g) * 16);
          if constexpr (I8) {
            const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, hi[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t a0, a1, a2, a3;
              s8x4_to_f16x2x2(lo[i], a0, a2);
              s8x4_to_f16x2x2(hi[i], a1, a3);
              mma_f16_16816(part[mt], a0, a1, a2, a3, b[2 * i], b[2 * i + 1]);
            }
          } else {
            mma_bf16_16816(part[mt], w0.x, w1.x, w0.y, w1.y, b[0], b[1]);
            mma_bf16_16816(part[mt], w0.z, w1.z, w0.w, w1.w, b[2], b[3]);
          }
        }
      }
    }
    const bool last = n.u == v1;
    if (last || n.kb == 0 || (I8 && ++folded == 8)) {  // 8-bit: at most 1024 k, sums of at most 2^24
      fold();
      folded = 0;
      if (!last && n.kb == 0 && n.a == 0) {
        finish(c.tile);
        first_u = n.u;
      }
      c = n;
      if (!last && n.kb == 0) enter();
    }
    c = n;
  }
  __syncthreads();

  // ---------------------------------------------------------------- tiles that warps or CTAs share
  // 0: the part of a tile that began in an earlier CTA, 1: of one that ends in a later CTA
  auto slot_of = [&](int cta, int tail) { return p.slots + ((int64_t)cta * 2 + tail) * (p.M * R); };
  const int tile0 = u0 / whole, tile1 = u1 > u0 ? (u1 - 1) / whole : tile0 - 1;
#pragma unroll 1
  for (int tile = tile0; tile <= tile1; ++tile) {
    const int s = tile * whole, e = s + whole, a = max(s, u0), b = min(e, u1);
    // the warps that hold parts of it
    int lo = 0, hi = W - 1;
    while (bound(lo + 1) <= a) ++lo;
    while (bound(hi) >= b) --hi;
    if (lo == hi && a == s && b < bound(lo + 1)) continue;  // written: whole, and not the warp's last
#pragma unroll 1
    for (int i = threadIdx.x; i < p.M * R; i += THREADS) {
      float v = 0.f;
#pragma unroll 1
      for (int w = lo; w <= hi; ++w) {
        const int end = bound(w + 1);
        if (bound(w) == end) continue;
        v += end <= e ? s_y[w * ysize + i / R * kPitch + i % R] : __ldcg(head_of(w) + i);
      }
      if (a > s || b < e)
        __stcg(slot_of(blockIdx.x, a == s) + i, v);
      else
        put(tile, i, v);
    }
  }
  // At most two tiles, the first and the last, have parts in other CTAs: the last CTA of each adds the
  // parts in the order of K
  const bool cut0 = tile0 <= tile1 && (tile0 * whole < u0 || (tile0 + 1) * whole > u1);
  const bool cut1 = tile1 > tile0 && (tile1 + 1) * whole > u1;
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 64 && lane == 0) {
    const int tile = warp ? tile1 : tile0;
    bool last = false;
    if (warp ? cut1 : cut0) {
      const int c0 = tile * whole / share, c1 = ((tile + 1) * whole - 1) / share;
      last = atomicAdd(p.tickets + c0, 1u) == (unsigned)(c1 - c0);
      if (last) p.tickets[c0] = 0u;
    }
    s_last[warp] = last;
  }
  if (I8 && threadIdx.x == 64) {
    // every CTA has read h's maxima before its first product: the last one here leaves them zero
    s_last[2] = atomicAdd(p.tickets + gridDim.x, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (I8 && s_last[2]) {
    for (int i = threadIdx.x; i < P; i += THREADS) p.amax[i] = 0u;
    if (threadIdx.x == 0) p.tickets[gridDim.x] = 0u;
  }
  if (!s_last[0] && !s_last[1]) return;
  __threadfence();  // the other parts were fenced before their counts
  const int quads = p.M * (R / 4);  // four rows of a token each
#pragma unroll 1
  for (int i = threadIdx.x; i < 2 * quads; i += THREADS) {
    const int which = i >= quads, at = i - which * quads;
    if (!s_last[which]) continue;
    const int tile = which ? tile1 : tile0;
    put4<R>(p, tile, at, add_parts(slot_of, tile * whole / share, ((tile + 1) * whole - 1) / share, at));
  }
}

template <int FMT, int DEPTH, bool FINE, bool ZP>
cudaError_t launch_gu(const StreamArgs& a, int x_bytes, int depth, cudaStream_t st) {
  auto* kfn = gate_up_kernel<FMT, DEPTH, FINE, ZP>;
  static OncePerDevice once;
  if (const cudaError_t e = raise_smem_limit(kfn, once); e != cudaSuccess) return e;
  const int P = a.M * a.topk;
  const int lists = gu_list_bytes(P);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kNumSMs, 1, 1);
  cfg.blockDim = dim3(kGuWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = (size_t)(x_bytes + lists + kGuWarps * depth * kStage);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, a, x_bytes, lists, depth);
}

template <int FMT, int W, bool FINE, bool ZP>
cudaError_t launch_dn(const StreamArgs& a, cudaStream_t st) {
  auto* kfn = down_kernel<FMT, W, FINE, ZP>;
  static OncePerDevice once;
  if (const cudaError_t e = raise_smem_limit(kfn, once); e != cudaSuccess) return e;
  const int P = a.M * a.topk;
  const int lists = (W * a.M * (kDnRows + 4) * 4 + P * (int)(sizeof(Entry) + 2 * 4 + 2 * 2) + 127) & ~127;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kNumSMs, 1, 1);
  cfg.blockDim = dim3(W * 32, 1, 1);
  cfg.dynamicSmemBytes = (size_t)kSmem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, a, lists);
}

// Warps of DOWN: what leaves each a ring of two stages with 8 tokens beside the results of all.  4-bit
// weights are bound by instructions and take more: at 12 tokens 16 and 12 warps take 13.4 and 14.4 us on 8
// experts of 512x1024 and are even on 60 of 1376x2080.  Of bf16 and 8-bit weights 16 warps make
// nothing of one to 8 tokens faster (47.7 and 48.2 us, 485.9 and 488.2 us, 36.9 and 35.9 us).
template <int FMT>
__host__ __device__ constexpr int dn_warps(int tokens) {
  return FMT != STREAM_INT4 ? 8 : tokens <= kDnFew ? 16 : 12;
}
template <int FMT>
constexpr bool dn_fits(int tokens) {
  constexpr int WB = FMT == STREAM_INT4 ? 64 : 128, XB = FMT == STREAM_BF16 ? 128 : 256;
  const int stage = kDnRows * WB + 8 * XB;
  return dn_warps<FMT>(tokens) * (tokens * (kDnRows + 4) * 4 + 2 * stage) + tokens * kMoeMaxTopk * 20 + 128 <= kSmem;
}
static_assert(dn_fits<STREAM_INT4>(kDnFew) && dn_fits<STREAM_INT4>(kMoeMaxTokens) && dn_fits<STREAM_INT8>(kMoeMaxTokens),
              "two stages for every warp");

template <int FMT, bool FINE, bool ZP>
cudaError_t launch_dn_warps(const StreamArgs& a, cudaStream_t st) {
  if (FMT == STREAM_INT4 && a.M <= kDnFew) return launch_dn<FMT, dn_warps<FMT>(kDnFew), FINE, ZP>(a, st);
  return launch_dn<FMT, dn_warps<FMT>(kMoeMaxTokens), FINE, ZP>(a, st);
}

// bytes of GATE_UP's tokens in shared memory
int64_t gu_x_bytes(int fmt, const StreamArgs& a) {
  const int64_t ks = gu_k(fmt), stages = (a.K + ks - 1) / ks;
  return (stages * ks * 2 * a.M + 127) & ~int64_t(127);
}

// stages of GATE_UP's rings beside the tokens
int gu_depth(int fmt, const StreamArgs& a) {
  const int64_t left = kSmem - gu_x_bytes(fmt, a) - gu_list_bytes(a.M * a.topk);
  return left < 0 ? 0 : (int)std::min<int64_t>(kGuDepth, left / (kGuWarps * kStage));
}

template <bool FINE, bool ZP>
cudaError_t launch_gu_int4(const StreamArgs& a, int x, int depth, cudaStream_t st) {
  if (depth == kGuDepth) return launch_gu<STREAM_INT4, kGuDepth, FINE, ZP>(a, x, depth, st);
  return launch_gu<STREAM_INT4, 0, FINE, ZP>(a, x, depth, st);
}

}  // namespace

// 4-bit weights: rings of two or three stages too.  8 of 256 experts of 2048x4096, this kernel and
// stream_kernel: 12 tokens (3 stages) 208 and 280 us, 18 tokens (2 stages) 299 and 373 us; bf16: 15
// tokens (3) 747 and 707 us, 18 tokens (2) 984 and 801 us; 8-bit: 18 tokens (2) 522 and 459 us.
bool gate_up_few_takes(int fmt, const StreamArgs& a) { return gu_depth(fmt, a) >= (fmt == STREAM_INT4 ? 2 : kGuDepth); }

cudaError_t launch_gate_up_few(int fmt, const StreamArgs& a, cudaStream_t st) {
  const int x = (int)gu_x_bytes(fmt, a), d = gu_depth(fmt, a);
  if (fmt == STREAM_BF16) return launch_gu<STREAM_BF16, kGuDepth, false, false>(a, x, d, st);
  if (fmt == STREAM_INT8) return launch_gu<STREAM_INT8, kGuDepth, false, false>(a, x, d, st);
  if (a.group_shift < 7)
    return a.zero ? launch_gu_int4<true, true>(a, x, d, st) : launch_gu_int4<true, false>(a, x, d, st);
  return a.zero ? launch_gu_int4<false, true>(a, x, d, st) : launch_gu_int4<false, false>(a, x, d, st);
}

cudaError_t launch_down(int fmt, const StreamArgs& a, cudaStream_t st) {
  if (fmt == STREAM_BF16) return launch_dn_warps<STREAM_BF16, false, false>(a, st);
  if (fmt == STREAM_INT8) return launch_dn_warps<STREAM_INT8, false, false>(a, st);
  if (a.group_shift < 7)
    return a.zero ? launch_dn_warps<STREAM_INT4, true, true>(a, st) : launch_dn_warps<STREAM_INT4, true, false>(a, st);
  return a.zero ? launch_dn_warps<STREAM_INT4, false, true>(a, st) : launch_dn_warps<STREAM_INT4, false, false>(a, st);
}

size_t down_head_bytes(int64_t M) {
  return (size_t)kNumSMs * dn_warps<STREAM_INT4>((int)M) * M * kDnRows * 4;  // the most of all types
}

}  // namespace ql
