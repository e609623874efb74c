// Linear layers on 4-bit integer weights with group scales, for few tokens: y = x W^T, and the gated
// block h = silu(a min(g, L)) clamp(u, -L, L) on such weights, streaming them once per 32 tokens.
//
//   w[n,k] = (q[n,k] - z[n,k/G]) * s[n,k/G],   q in 0..15, z in 0..255 (8 without zero points)
//   y[m,n] = bf16( sum_groups s * sum_{k in group} x[m,k] (q - z) )      (+ bias after the cast)
//
// q - z is exact in bf16 and a bf16 product is exact in fp32, so the warp MMA (bf16 operands, fp32
// sums) adds exact products and each group's sum is multiplied by its scale once, in fp32: no
// weight is rounded.
//
// The weights are the MMA's A operand, the tokens its columns.  A warp owns 32 rows of W (a gated
// block: 16 gate rows and the 16 up rows of the same outputs, so that one lane holds both sums of
// an output) and walks K in blocks of 128, 64 bytes of every row, through a ring of its own that it
// fills with cp.async: warps need no barrier between them.  Which k an MMA slot stands for is free
// as long as both operands agree, so the codes stay in the order in which a word's nibbles come out
// in pairs, and the activations are put in that order (pair_up).  The activations travel in the same
// ring as the weights that meet them; one token of many rows is staged for a whole CTA instead.
//
// What bounds it: a block of 16 rows takes about 150 warp instructions, half of them on the ALU,
// which takes one every two cycles, from two to six warps per scheduler that each run a dependent
// chain: with the loads taken out, 1 x 17408 x 5120 (gated) still takes 17.4 us; with the
// arithmetic taken out 18.1 us; both together 22.2 us (4.2 TB/s; HBM alone 13.7).  1 x 5120 x 17408
// 17.2 us (2.7 TB/s), 8 tokens 18.9; 16 x 10240 x 5120 with groups of 32 15.4 us.  Two row tiles a
// warp against one: two independent MMA chains, and the activations are read once for both (28.2
// to 23.6 us).  Scales a step ahead, shared by shuffles: 2-byte loads waited for in the block that
// uses them took 11 us of 35.
#include <cuda_fp16.h>


#include "common.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "internal.h"

namespace ql {

namespace {

constexpr int kBlockK = 128;
constexpr int kRowTiles = 2;  // of 16 rows, a warp
constexpr int kPrefetch = 2;  // steps

struct Plan {
  int chunk;    // staged activations: blocks of K at a time
  int x_bytes;  // of them
  int kw;       // warps of a row group
};
// bytes of a block of staged activations
__host__ __device__ constexpr uint32_t x_block(bool fine) { return fine ? 256 : 320; }

// bf16 bit patterns below 256 are linear, pattern p has the value p 2^-133 (subnormals, then the
// first binade), so a nibble left in bits 0..3 or 4..7 of a half word already is q 2^-133 or
// q 2^-129: one multiply-add, exact, turns it into (q - z) / 64.  Against the usual 128 + q (a
// shift, an AND-OR and a subtraction per pair) this drops two of three shifts per word; the ALU
// takes a warp's integer instruction every two cycles and bounds these kernels.
constexpr uint32_t kLoMul = 0x7F007F00u;   // bf16x2 of 2^127
constexpr uint32_t kHiMul = 0x7D007D00u;   // bf16x2 of 2^123
constexpr uint32_t kNegMul = 0xFF00FF00u;  // bf16x2 of -2^127: a zero point's pattern to -z / 64

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// the eight codes of a word as bf16x2 of (q - z) / 64: (e0,e4) (e1,e5) (e2,e6) (e3,e7)
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t negz, uint32_t (&o)[4]) {
  const uint32_t v = w >> 8;
  o[0] = fma_bf16x2(w & 0x000F000Fu, kLoMul, negz);
  o[1] = fma_bf16x2(w & 0x00F000F0u, kHiMul, negz);
  o[2] = fma_bf16x2(v & 0x000F000Fu, kLoMul, negz);
  o[3] = fma_bf16x2(v & 0x00F000F0u, kHiMul, negz);
}
// eight activations in the order of the codes
__device__ __forceinline__ uint4 pair_up(uint4 x) {
  return make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                    __byte_perm(x.y, x.w, 0x7632));
}
__device__ __forceinline__ float scale_to_f32(uint16_t bits, int fp16) {
  return fp16 ? __half2float(__ushort_as_half(bits)) : bf16_bits_to_f32(bits);
}
// the first MMA of a group's sum: no accumulator to clear
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory; zeros, and no access to src, where `take` is 0
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
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_cta(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

// NT: 8-token tiles; FINE: groups shorter than 128; ZP: zero points given; XS: one token, staged for
// the CTA, else the activations travel in the warps' rings; SEG: bytes of a row that a step copies;
// kDepth: steps in a ring; W: warps, on RW row groups; the warps of a row group, two at least, split K.
// gridDim.z CTAs (a cluster) take contiguous shares of K.
// Up to 8 tokens the compiler is told that 16 warps share an SM, 128 registers a thread: left alone it
// used 72 to 127 and ran 2 to 7 % longer (gated 1 x 10240 x 5120 21.7 us, so 20.5; int4 2 x 5120 x
// 17408, groups of 64, 19.2 and 18.6); with more tokens the same bound costs 10 to 57 %.
template <bool GATED, int NT, bool FINE, bool ZP, bool XS, int SEG, int kDepth, int W, int RW>
__global__ void __launch_bounds__(W * 32, NT > 1 || (XS && FINE && ZP) ? 0 : 16 / W)
    int4_kernel(const __grid_constant__ FfnSkinnyArgs a, const Plan p) {
  constexpr int kThreads = W * 32, MT = kRowTiles;
  constexpr int TT = NT * 8, RT = MT * 16, OUT = GATED ? RT / 2 : RT, PITCH = TT + 1;
  constexpr int SB = SEG / 64;                   // blocks per step
  constexpr int LPR = SEG / 16, RPI = 32 / LPR;  // lanes per row, rows per copy instruction
  constexpr uint32_t kX = RT * SEG;                   // weight bytes of a warp's step
  constexpr uint32_t kStep = kX + (XS ? 0 : TT * 256);  // all of its bytes
  static_assert(XS || SB == 1, "activations: one block per step");
  constexpr uint32_t XB = x_block(FINE);
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem + p.x_bytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  constexpr int KW = W / RW;
  static_assert(KW > 1 && KW * RW == W, "the sums meet in shared memory");
  const int wr = warp % RW, wk = warp / RW;
  // (one staged token, groups shorter than 128, zero points: with the warps' stride known and the
  // register bound above the compiler's order of the loop took 1 x 16000 x 17408 64.7 us, so 51.0)
  const int kw = XS && FINE && ZP ? p.kw : KW;
  const int m0 = blockIdx.y * TT, toks = min(TT, a.M - m0);
  const int n_cta = (int)blockIdx.x * RW * OUT, n0 = n_cta + wr * OUT;
  const int ks = gridDim.z, kz = blockIdx.z;
  const int nblk = (a.K + kBlockK - 1) / kBlockK;
  const int c0 = nblk / ks * kz + min(kz, nblk % ks), c1 = c0 + nblk / ks + (kz < nblk % ks);
  const uint32_t mine = smem_addr(ring) + (uint32_t)warp * (kDepth * kStep);

  // copies: lane = (row of RPI, 16-byte piece of the segment).  Piece c of row r lies in slot
  // c ^ f(r), f(r) = (r % 2) * 4 + r / 2 % 4: reading four pieces of two rows (LDS.128) or one word
  // of a piece of eight rows (FINE) meets every bank once.  Rows of a gated block: all gate rows,
  // then all up rows
  const int cr = lane / LPR, cc = lane % LPR;
  auto swz = [](int r) { return (((r & 1) << 2) | ((r >> 1) & 3)) & (LPR - 1); };
  const int valid = min(OUT, a.N - n0);  // outputs that exist
  const uint8_t* wp = a.w + (int64_t)(n0 + cr) * a.ldw_bytes + (int64_t)(c0 + wk * SB) * 64 + cc * 16;
  const int64_t rstep = (int64_t)RPI * a.ldw_bytes;
  const int64_t to_up = ((int64_t)a.N - OUT) * a.ldw_bytes;
  // activations in the ring: a row of 16 pieces per token, lane = (row of two, piece).  Piece c of
  // token m lies in slot c ^ h, FINE: h = 4 (m % 2), else h = c / 8 + 2 (m % 2): four lanes of a token
  // and four of the next then meet every bank once.  Read where they are used, the loads took 6 of 18
  // us at 16 x 10240 x 5120 (15.0 so; 8 x 5120 x 17408 21.6 to 19.2 us, 32 tokens 60 to 42 us)
  const int xc = lane & 15, xm = lane >> 4;
  const uint16_t* xq = a.x + (int64_t)(m0 + xm) * a.ldx + (int64_t)(c0 + wk * SB) * kBlockK + xc * 8;
  const uint32_t x_dst = kX + (uint32_t)(xm * 256 + (xc ^ (FINE ? xm * 4 : (xc >> 3) + xm * 2)) * 16);
  int bf = c0 + wk * SB;  // first block of the next step to copy
  auto fetch = [&](uint32_t slot) {
    if (bf < c1) {
      // past the share's end: another CTA's blocks or the row's padding, not copied
      const bool in = bf + (cc >> 2) < c1 && bf * kBlockK + cc * 32 < a.K;
      const uint8_t* src = wp;
      const uint32_t dst = mine + slot * kStep + (uint32_t)(cr * SEG + ((cc ^ swz(cr)) * 16));
#pragma unroll
      for (int i = 0; i < RT / RPI; ++i) {
        if (GATED && i * RPI == OUT) src += to_up;
        const int r = i * RPI + cr;
        // rows a multiple of eight apart share f; RPI = 4, 2: the later rows' f differs in known bits
        const uint32_t flip = (uint32_t)((swz(i * RPI)) * 16);
        cp16((dst ^ flip) + i * RPI * SEG, src, in && (GATED && i * RPI >= OUT ? r - OUT : r) < valid);
        src += rstep;
      }
      if constexpr (!XS) {
        const uint16_t* xs = xq;
        const bool in = bf * kBlockK + xc * 8 < a.K;
#pragma unroll
        for (int i = 0; i < TT / 2; ++i) {
          cp16(mine + slot * kStep + x_dst + i * 512, xs, in && i * 2 + xm < toks);
          xs += 2 * a.ldx;
        }
        xq += kw * kBlockK;
      }
      wp += kw * SEG;
      bf += kw * SB;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Before the wait for the launch before, nothing is read or written but L2 is asked for the first
  // steps' rows (a prefetch only moves them there): a row per lane
  {
    const int o = GATED ? lane % OUT : lane;
    if (o < valid) {
      const uint8_t* row = a.w + ((GATED && lane >= OUT ? (int64_t)a.N : 0) + n0 + o) * a.ldw_bytes;
      for (int d = 0, b = c0 + wk * SB; d < kPrefetch && b < c1; ++d, b += kw * SB) prefetch_l2(row + (int64_t)b * 64);
    }
  }
  pdl_wait();
  // staged activations of a chunk.  All CTAs read the same few lines of L2, which serves a line's
  // requests one after the other: whole lines are asked for (with neighbouring lanes 64 bytes apart
  // this took 5 us more at 1 x 17408 x 5120).  Piece 4 t + j of a block lies at 80 t + 16 j, so that
  // the four lanes meet every bank once; FINE lanes read neighbouring pieces.  Every thread then puts
  // its own pieces in the order of the codes
  auto x_slot = [](int i) { return (uint32_t)(FINE ? i * 16 : (i >> 4) * XB + ((i >> 2) & 3) * 80 + (i & 3) * 16); };
  auto x_copy = [&](int q0, int q1) {
    const uint16_t* src = a.x + (int64_t)m0 * a.ldx + (int64_t)q0 * kBlockK;
    for (int i = threadIdx.x; i < (q1 - q0) * 16; i += kThreads)
      cp16(smem_addr(smem) + x_slot(i), src + i * 8, q0 * kBlockK + i * 8 < a.K);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto x_order = [&](int q0, int q1) {
    for (int i = threadIdx.x; i < (q1 - q0) * 16; i += kThreads) {
      uint4* at = reinterpret_cast<uint4*>(smem + x_slot(i));
      *at = pair_up(*at);
    }
  };
  if constexpr (XS) x_copy(c0, min(c0 + p.chunk, c1));
#pragma unroll 1
  for (int d = 0; d < kDepth - 1; ++d) fetch(d);

  // scales and zero points of a step's blocks, read one step ahead and kept as read (converting
  // them at once would wait for the loads).  The four lanes of a row share them: lane t reads
  // those of block t of four, FINE: those of piece t of every block, and shuffles hand them out
  constexpr int SL = FINE ? SB : (SB + 3) / 4;
  uint16_t s_next[SL][MT][2];
  uint8_t z_next[SL][MT][2];
  const uint16_t* sp[MT][2];
  const uint8_t* zp[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int n = n0 + (GATED ? mt * 8 : mt * 16 + 8 * h) + g;
      if (n >= a.N) n = a.N - 1;
      const int64_t row = GATED && h ? (int64_t)a.N + n : n;
      sp[mt][h] = a.scale + row * a.lds;
      zp[mt][h] = ZP ? a.zero + row * a.ldz : nullptr;
    }
  auto scales = [&](int b0) {
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int k = (b0 + (FINE ? i : i * 4 + t % SB)) * kBlockK + (FINE ? 32 * t : 0);
      const int gi = min(k, a.K - 1) >> a.group_shift;  // past the end: any, its x is zero
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (FINE: a group past the end has no scale, its sum of zeros stays zero)
          s_next[i][mt][h] = FINE && k >= a.K ? (uint16_t)0 : sp[mt][h][gi];
          if (ZP) z_next[i][mt][h] = zp[mt][h][gi];
        }
    }
  };
  scales(min(c0 + wk * SB, nblk - 1));

  float acc[MT][NT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;

  // this lane's pieces of its token: staged (every lane of a row of the MMA reads the one token), or
  // in a ring's slot
  const uint32_t x_at = smem_addr(smem) + (uint32_t)(FINE ? t * 16 : t * 80);
  const uint32_t x_src = (uint32_t)((FINE ? t ^ (g & 1) << 2 : t * 4 ^ (t >> 1 | (g & 1) << 1)) * 16);
  const uint32_t negz8 = 0xBE00BE00u;  // bf16x2 of -8 / 64
  uint32_t slot = 0;
  for (int q0 = c0; q0 < c1; q0 += XS ? p.chunk : c1 - c0) {
    const int q1 = XS ? min(q0 + p.chunk, c1) : c1;
    if constexpr (XS) {
      if (q0 == c0) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      } else {
        __syncthreads();  // the chunk before is read
        x_copy(q0, q1);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      x_order(q0, q1);
      __syncthreads();
    }

    for (int b0 = q0 + wk * SB; b0 < q1; b0 += kw * SB) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
      __syncwarp();  // every lane's copies of this step have landed, and the step before is read
      fetch(slot == 0 ? kDepth - 1 : slot - 1);
      const uint32_t from = mine + slot * kStep + (uint32_t)(g * SEG);
      const uint32_t x_from = mine + slot * kStep + kX + (uint32_t)(g * 256);
      if (++slot == kDepth) slot = 0;
      // 64 x scale and the zero point in one word: a bf16 or fp16 scale leaves the low 13 bits of
      // its fp32 image free
      uint32_t sz[SL][MT][2];
#pragma unroll
      for (int i = 0; i < SL; ++i)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            sz[i][mt][h] = __float_as_uint(scale_to_f32(s_next[i][mt][h], a.scale_fp16) * 64.f) |
                           (ZP ? z_next[i][mt][h] : 0u);
      if (b0 + kw * SB < c1) scales(b0 + kw * SB);
#pragma unroll
      for (int sb = 0; sb < SB; ++sb) {
        if (sb > 0 && b0 + sb >= q1) break;
        uint32_t wv[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t tile = from + (GATED ? mt * 8 + h * OUT : mt * 16 + h * 8) * SEG;
            if constexpr (FINE) {
              // word t of every 32-k piece, so that an MMA stays inside one group
#pragma unroll
              for (int j = 0; j < 4; ++j) wv[mt][h][j] = lds4(tile + ((sb * 4 + j) ^ swz(g)) * 16 + t * 4);
            } else {
              const uint4 v = lds16(tile + ((sb * 4 + t) ^ swz(g)) * 16);
              wv[mt][h][0] = v.x;
              wv[mt][h][1] = v.y;
              wv[mt][h][2] = v.z;
              wv[mt][h][3] = v.w;
            }
          }
        const uint32_t x_block0 = x_at + (uint32_t)(b0 + sb - q0) * XB;
        uint32_t negz[MT][2];
        float sc[MT][2], part[MT][NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j == 0 || FINE) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t v = FINE ? __shfl_sync(0xffffffffu, sz[FINE ? sb : 0][mt][h], j, 4)
                                        : __shfl_sync(0xffffffffu, sz[FINE ? 0 : sb / 4][mt][h], sb & 3, 4);
                sc[mt][h] = __uint_as_float(ZP ? v & ~255u : v);
                negz[mt][h] = ZP ? fma_bf16x2(__byte_perm(v, 0u, 0x4040), kNegMul, 0u) : negz8;
              }
          }
          uint4 bx[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            bx[nt] = XS ? lds16(x_block0 + j * (FINE ? 64 : 16))
                        : pair_up(lds16(x_from + nt * 2048 + (x_src ^ (uint32_t)(j * (FINE ? 64 : 16)))));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t q0v[4], q1v[4];
            codes_to_bf16(wv[mt][0][j], negz[mt][0], q0v);
            codes_to_bf16(wv[mt][1][j], negz[mt][1], q1v);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (j == 0 || FINE)
                mma_first(part[mt][nt], q0v[0], q1v[0], q0v[1], q1v[1], bx[nt].x, bx[nt].y);
              else
                mma_bf16_16816(part[mt][nt], q0v[0], q1v[0], q0v[1], q1v[1], bx[nt].x, bx[nt].y);
              mma_bf16_16816(part[mt][nt], q0v[2], q1v[2], q0v[3], q1v[3], bx[nt].z, bx[nt].w);
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
  }

  // the next launch may take the places that become free (asked for earlier, its CTAs took places
  // unevenly while this launch ran: 16 x 10240 x 5120 21.0 against 18.9 us)
  pdl_launch_dependents();
  auto store = [&](float v, float u, int m, int n) {
    uint16_t yb;
    if constexpr (GATED) {
      yb = f32_to_bf16_rn(gated_act(v, u, a.alpha, a.limit));
    } else {
      yb = f32_to_bf16_rn(v);
      if (a.bias) yb = f32_to_bf16_rn(bf16_bits_to_f32(yb) + bf16_bits_to_f32(a.bias[n]));
    }
    a.y[(int64_t)(m0 + m) * a.ldy + n] = yb;
  };
  // every warp leaves its sums in its own part of the ring (its copies have landed and are read).
  // Accumulator i of lane (g, t): row g + 8 (i >> 1), token 2t + (i & 1)
  static_assert(RT * PITCH * 4 <= kDepth * kStep, "a warp's sums fit its part of the ring");
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
  auto sums = [&](int w) { return reinterpret_cast<float*>(ring + w * (kDepth * kStep)); };
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sums(warp)[(mt * 16 + g + 8 * (i >> 1)) * PITCH + nt * 8 + 2 * t + (i & 1)] = acc[mt][nt][i];
  __syncthreads();
  if (ks > 1) {
    // the K shares of this CTA into the first one's place: each value has one reader and writer
    for (int e = threadIdx.x; e < RW * RT * toks; e += kThreads) {
      const int r = e % RT, w = e / RT % RW, m = e / (RT * RW);
      float v = 0.f;
      for (int i = 0; i < KW; ++i) v += sums(w + i * RW)[r * PITCH + m];
      sums(w)[r * PITCH + m] = v;
    }
    __syncthreads();
  }
  if (ks > 1) cluster_sync_all();
  auto total = [&](int w, int r, int m) {
    float v = 0.f;
    if (ks == 1) {
      for (int i = 0; i < KW; ++i) v += sums(w + i * RW)[r * PITCH + m];
    } else {
      for (int z = 0; z < ks; ++z) v += ld_cta(smem_addr(sums(w) + r * PITCH + m), (uint32_t)z);
    }
    return v;
  };
  // the CTAs of a cluster share the outputs
  for (int e = kz * kThreads + threadIdx.x; e < RW * OUT * toks; e += ks * kThreads) {
    const int o = e % (RW * OUT), m = e / (RW * OUT), w = o / OUT, oo = o % OUT;
    const int r = GATED ? (oo >> 3) * 16 + (oo & 7) : oo;
    if (n_cta + o < a.N) store(total(w, r, m), GATED ? total(w, r + 8, m) : 0.f, m, n_cta + o);
  }
  if (ks > 1) cluster_sync_all();  // the others may still read this CTA's sums
}

template <bool GATED, int NT, bool FINE, bool ZP, bool XS, int SEG, int kDepth, int W, int RW>
cudaError_t launch(const FfnSkinnyArgs& a, cudaStream_t st) {
  constexpr int MT = kRowTiles, out = (GATED ? MT * 8 : MT * 16) * RW, kw = W / RW;
  auto* kfn = int4_kernel<GATED, NT, FINE, ZP, XS, SEG, kDepth, W, RW>;
  static OncePerDevice once;
  if (const cudaError_t e = raise_smem_limit(kfn, once); e != cudaSuccess) return e;
  const int nblk = (a.K + kBlockK - 1) / kBlockK;
  Plan p = {};
  p.kw = kw;
  const int64_t tiles = (int64_t)((a.N + out - 1) / out) * ((a.M + NT * 8 - 1) / (NT * 8));
  // K over a cluster's CTAs while eight warps per SM are missing and every warp keeps four blocks or
  // more (1 x 5120 x 17408: 2 CTAs 17.1 us, 1: 20.7, 4: 19.7; 16 x 4096 x 4096: 1: 5.6, 2: 10.2, 4: 17.8)
  int ks = 1;
  while (ks < 8 && tiles * ks * W < 8 * kNumSMs && nblk >= kw * ks * 8) ks *= 2;
  if constexpr (XS) {
    // the activations of the CTA's share of K, or of as many blocks of it as 32 KB hold
    constexpr int xb = (int)x_block(FINE);
    const int step = SEG / 64 * kw;
    const int share = ((nblk + ks - 1) / ks + step - 1) / step * step;
    p.chunk = 32 * 1024 / xb / step * step;
    if (p.chunk > share) p.chunk = share;
    p.x_bytes = (p.chunk * xb + 127) & ~127;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + out - 1) / out), (unsigned)((a.M + NT * 8 - 1) / (NT * 8)), (unsigned)ks);
  cfg.blockDim = dim3(W * 32, 1, 1);
  cfg.dynamicSmemBytes = (size_t)W * kDepth * (MT * 16 * SEG + (XS ? 0 : NT * 8 * 256)) + p.x_bytes;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 1;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = (unsigned)ks;
  cfg.attrs = at;
  cfg.numAttrs = ks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kfn, a, p);
}

template <bool GATED, bool FINE, bool ZP>
cudaError_t launch_nt(const FfnSkinnyArgs& a, cudaStream_t st) {
  // row tiles of a warp, for 32 tokens; up to one per SM, more warps share a tile's K in place of more
  // CTAs
  const int64_t tiles = (int64_t)((a.N + (GATED ? 15 : 31)) / (GATED ? 16 : 32)) * ((a.M + 31) / 32);
  const bool few = tiles <= kNumSMs;
  // One token of many rows is staged: 1 x 5120 x 17408 17.1 us, in the rings 18.9.  From four tiles
  // per SM on, eight warps on four row groups share it (1 x 17408 x 5120 gated: 22.2 us against 25.8
  // with four warps on one row group; 1 x 14336 x 5120, 448 tiles: 13.2 and 12.8)
  if (a.M == 1 && tiles >= 4 * kNumSMs) return launch<GATED, 1, FINE, ZP, true, 128, 3, 8, 4>(a, st);
  if (a.M == 1 && !few) return launch<GATED, 1, FINE, ZP, true, 128, 3, 4, 1>(a, st);
  // 6 x 4096 x 4096: 16 warps 4.7 us, 8: 5.1, 4: 5.8; 6 x 5120 x 17408: 22.0, 20.2, 17.9; 16 warps want
  // two blocks each (6 x 512 x 1024, half of them idle: 2.0 us, 8 warps 2.0)
  if (a.M <= 8) {
    if (few && a.K > 31 * kBlockK) return launch<GATED, 1, FINE, ZP, false, 64, 3, 16, 1>(a, st);
    if (few) return launch<GATED, 1, FINE, ZP, false, 64, 3, 8, 1>(a, st);
    return launch<GATED, 1, FINE, ZP, false, 64, 3, 4, 1>(a, st);
  }
  // 13 x 2048 x 4096 gated: 8 warps 5.5 us, 4: 6.9; 16 x 10240 x 5120, groups of 32: 20.5 and 15.4
  if (a.M <= 16) {
    if (few) return launch<GATED, 2, FINE, ZP, false, 64, 3, 8, 1>(a, st);
    return launch<GATED, 2, FINE, ZP, false, 64, 2, 4, 1>(a, st);
  }
  // 25 x 2048 x 4096 gated: 8 warps 8.1 us, 4: 9.2; 32 x 10240 x 5120: 4 warps 22.7 us, 2: 23.3; 24 x
  // 17408 x 5120 gated: 53.4 and 50.7 (registers and shared memory leave room for 8 and 10 warps)
  if (few) return launch<GATED, 4, FINE, ZP, false, 64, 2, 8, 1>(a, st);
  if (tiles >= 4 * kNumSMs) return launch<GATED, 4, FINE, ZP, false, 64, 2, 2, 1>(a, st);
  return launch<GATED, 4, FINE, ZP, false, 64, 2, 4, 1>(a, st);
}

template <bool GATED>
cudaError_t launch_fmt(const FfnSkinnyArgs& a, cudaStream_t st) {
  if (a.group_shift < 7) return a.zero ? launch_nt<GATED, true, true>(a, st) : launch_nt<GATED, true, false>(a, st);
  return a.zero ? launch_nt<GATED, false, true>(a, st) : launch_nt<GATED, false, false>(a, st);
}

}  // namespace

cudaError_t launch_int4(bool gated, const FfnSkinnyArgs& a, cudaStream_t st) {
  return gated ? launch_fmt<true>(a, st) : launch_fmt<false>(a, st);
}

}  // namespace ql
