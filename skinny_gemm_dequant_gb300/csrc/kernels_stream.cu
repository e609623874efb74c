// Weight-streaming kernel for few tokens: gate and up of a mixture-of-experts layer whose tokens do not
// fit in shared memory (bf16, 8-bit and 4-bit weights), and the linear on 8-bit codes of few tokens.
//
//   GATE_UP  g = W13[e][0:I] x_m, u = W13[e][I:2I] x_m for every routed pair (m, j) with expert e,
//            h = bf16( silu(a min(g, L)) clamp(u, -L, L) )
//   LINEAR   y = (acc x_s) w_s, acc = sum_k x_q w_q  (+ bias after the cast)
//
// 8-bit weights: GATE_UP's tokens are quantised here, scale = max|v| / 127 over the
// row, code = v / scale rounded half to even; products of codes are exact in fp32, sums
// below 2^24 too, and every 1024 k they move to int32: sums are exact.  4-bit weights: q - z is
// exact in bf16, a group's fp32 sum is multiplied by its scale once.
//
// Persistent, one CTA per SM.  Units of 64 weight rows (32 gate, 32 up) by 64 or 128 k are cut evenly
// over the CTAs and dealt to their warps in turn; a unit's weights and its tokens' part of x come through
// the warp's own ring (cp.async), weights as the warp MMA's A operand.  At the end of an item (a tile for
// one entry of 8 tokens) the warps leave their sums in a buffer, and one more warp adds them and
// makes the results, of a CTA's last item all warps.  Items that CTAs share are joined by the last of
// them, which finds all parts in the workspace and adds them in the order of K, all warps at once (by one warp
// 16 tokens of 2048x4096 took 25 us, now 8).  Nobody waits for another CTA.
//
// Bound by HBM where units are many: LINEAR 1x17408x5120 19.2 us (4.6 TB/s; 5 us of start, first
// loads and last join), 16 tokens 28 us, GATE_UP of 24 tokens, 8 of 256 experts of 2048x4096, with DOWN: bf16 982 us
// (7.0 TB/s), 8-bit 559 us (6.2 TB/s).  4-bit weights 475 us (3.7 TB/s): the chain of a unit's loads, nibbles,
// scales and products, three warps a scheduler.
// Tiles of 32 rows took 66 us where 64 take 55 (8-bit, one token): half the copies of x.  LINEAR's passes
// of 16 tokens over a tile follow each other in one CTA, so that only the first reads HBM (linear_streams).
#include <cuda_fp16.h>

#include "common.cuh"
#include "ffn_act.cuh"
#include "moe_dispatch.cuh"
#include "stream.h"
#include "stream_dev.cuh"

namespace ql {

namespace {

constexpr int R = kStreamRows;
constexpr int MT = R / 16;
constexpr int kPitch = R + 4;  // of a column of sums: lanes (g, t) write 8 t + g, all banks once
constexpr int kBuffers = 4;  // of sums, at most

__host__ __device__ constexpr int compute_warps(int fmt) { return fmt == STREAM_INT4 ? 11 : 8; }
__host__ __device__ constexpr int unit_k(int fmt) { return fmt == STREAM_BF16 ? 64 : 128; }
__host__ __device__ constexpr int row_bytes(int fmt) { return fmt == STREAM_INT4 ? 64 : 128; }
__host__ __device__ constexpr int token_bytes(int fmt, int mode) {
  return fmt == STREAM_BF16 || mode == STREAM_LINEAR ? 128 : 256;
}

// shared memory: lists, buffers of the warps' sums, the warps' rings.  Both of the latter are cut when
// the largest number of tokens that meet an expert's weights is known: most often it is 1 or 2 of 8
struct Layout {
  int lists, total;  // bytes
};
constexpr int kSmem = 227 * 1024 - 1024;
__host__ __device__ constexpr int list_bytes(int fmt, int pairs) {
  return (pairs * (int)(sizeof(Entry) + 4 + 2 * 2) + (fmt == STREAM_INT8 ? kMoeMaxTokens * 8 : 0) + 127) & ~127;
}
// stages of a warp's ring beside one buffer of sums, with `tokens` of an entry
constexpr int ring_stages(int fmt, int mode, int pairs, int tokens) {
  return (kSmem - list_bytes(fmt, pairs) - compute_warps(fmt) * tokens * kPitch * 4 - 128) /
         (compute_warps(fmt) * (R * row_bytes(fmt) + tokens * token_bytes(fmt, mode)));
}

template <int ID0, int THREADS>
__device__ __forceinline__ void bar_sync(int b) {
  asm volatile("bar.sync %0, %1;" ::"r"(ID0 + b), "n"(THREADS) : "memory");
}
template <int ID0, int THREADS>
__device__ __forceinline__ void bar_arrive(int b) {
  asm volatile("bar.arrive %0, %1;" ::"r"(ID0 + b), "n"(THREADS) : "memory");
}
// position of a warp in its CTA's units
struct Walk {
  int u, item, kb, a, tile;
  __device__ void set(int u_, int nblk, int entries) {
    u = u_;
    item = u / nblk;
    kb = u - item * nblk;
    tile = item / entries;
    a = item - tile * entries;
  }
  __device__ void next(int step, int nblk, int entries) {
    u += step;
    kb += step;
    while (kb >= nblk) {
      kb -= nblk;
      ++item;
      if (++a == entries) {
        a = 0;
        ++tile;
      }
    }
  }
};

template <int FMT, int MODE, int NT, bool FINE, bool ZP>
__global__ void __launch_bounds__((compute_warps(FMT) + 1) * 32, 1)
    stream_kernel(const __grid_constant__ StreamArgs p, const __grid_constant__ Layout lay) {
  constexpr int W = compute_warps(FMT), THREADS = (W + 1) * 32;
  constexpr int TT = NT * 8, KU = unit_k(FMT), WB = row_bytes(FMT), XB = token_bytes(FMT, MODE);
  constexpr bool GU = MODE == STREAM_GATE_UP, LIN = MODE == STREAM_LINEAR;
  constexpr bool I8 = FMT == STREAM_INT8, I4 = FMT == STREAM_INT4;
  static_assert(GU || I8, "the linear is on 8-bit codes");
  constexpr int kFull = 1, kEmpty = 1 + kBuffers;  // named barriers: a buffer of sums is written, is read
  constexpr int OUT = GU ? R / 2 : R;   // outputs of a tile: half gate rows, half up rows
  using Sum = typename std::conditional<I8, int, float>::type;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int P = LIN ? 0 : p.M * p.topk;

  // lists: entries, ids by pair, (INT8) factor and scale by token, sorted pairs and their tokens
  Lists l;
  l.entries = reinterpret_cast<Entry*>(smem);
  l.ids = reinterpret_cast<int*>(l.entries + P);
  float* s_inv = reinterpret_cast<float*>(l.ids + P);
  float* s_xs = s_inv + (I8 ? kMoeMaxTokens : 0);
  l.pair = reinterpret_cast<uint16_t*>(s_xs + (I8 ? kMoeMaxTokens : 0));
  l.tok = l.pair + P;
  l.keys = reinterpret_cast<int*>(smem + lay.lists);  // the rings are filled later
  l.heads = reinterpret_cast<Entry*>(l.keys + (P + 3) / 4 * 4);

  pdl_wait();
  pdl_launch_dependents();
  int ne, xt;  // entries, most tokens of one
  if constexpr (LIN) {
    ne = (p.M + TT - 1) / TT;
    xt = min(p.M, TT);
  } else {
    static_assert(TT == kPerEntry, "a token tile for each entry");
    route(p, l, W + 1);
    if (I8) {
#pragma unroll 1
      for (int m = W - warp; m < p.M; m += W + 1) {  // (from the last warp on: the first ones route)
        const uint4* row = reinterpret_cast<const uint4*>(p.x + m * p.ldx);
        float top = 0.f;
#pragma unroll 4
        for (int i = lane; i < p.K / 8; i += 32) {
          const uint4 v = row[i];
          const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            top = max_nan(max_nan(top, fabsf(__uint_as_float(q[j] << 16))), fabsf(__uint_as_float(q[j] & 0xFFFF0000u)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) {
          s_xs[m] = __fdiv_rn(top, 127.f);
          s_inv[m] = code_factor(top);
        }
      }
    }
    __syncthreads();
    ne = dispatch<W + 1>(p, l, kPerEntry, xt);
    // for the next launch
    if (blockIdx.x == gridDim.x - 1 && warp == W) hand_lists(p, l, ne, xt);
    if (blockIdx.x < p.M && warp == W) hand_weights(p, l, blockIdx.x);
  }
  const int buffer = W * xt * kPitch * 4, buffers = max(1, min(kBuffers, 24 * 1024 / buffer));
  const int rings = (lay.lists + buffers * buffer + 127) & ~127, stage = R * WB + xt * XB;
  const int depth = min(6, (lay.total - rings) / (W * stage));  // of a warp's ring; 2 at least (ring_stages)

  // ------------------------------------------------------------------ this CTA's units
  const int nblk = (p.K + KU - 1) / KU;
  const int tiles = (p.N + OUT - 1) / OUT;
  const int total = tiles * ne * nblk;
  const int share = unit_share(total, nblk, W);
  const int u0 = min(total, (int)blockIdx.x * share), u1 = min(total, u0 + share);

  auto entry = [&](int a) {
    if constexpr (LIN)
      return Entry{0, (uint16_t)(a * TT), min(TT, p.M - a * TT)};
    else
      return l.entries[a];
  };
  if (u0 >= u1) return;  // nothing was dispatched, or nothing is left
  const int item0 = u0 / nblk, item1 = (u1 - 1) / nblk;

  if (warp < W) {
    // ---------------------------------------------------------------- streaming and products
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_addr(smem) + (uint32_t)(rings + warp * depth * stage);
    constexpr int LPR = WB / 16, RPI = 32 / LPR;   // lanes per weight row, rows per copy
    constexpr int LPT = XB / 16, TPI = 32 / LPT;   // lanes per token row, tokens per copy
    constexpr int XCOPIES = TT / TPI;
    const int cr = lane / LPR, cc = lane % LPR, tr = lane / LPT, tc = lane % LPT;
    // piece c of row r lies in slot c ^ f(r): four pieces of two rows (LDS.128) or a word of a piece
    // of eight rows meet every bank once
    auto swz = [](int r) { return (((r & 1) << 2) | ((r >> 1) & 3)) & (LPR - 1); };
    const uint32_t w_dst = (uint32_t)(cr * WB + ((cc ^ swz(cr)) * 16));
    // slot of piece c of token m: the lanes of a read meet every bank once
    auto xswz = [](int c, int m) {
      if (XB == 128) return c ^ ((m & 1) << 2);
      if (I8) return c ^ (m & 1);
      return c ^ (FINE ? (m & 1) << 2 : (c >> 3) + ((m & 1) << 1));
    };

    Walk f;  // the next unit to copy
    f.set(u0 + warp, nblk, ne);
    int f_item = -1, f_valid = 0, f_toks = 0;
    const uint8_t* f_w = nullptr;
    const uint8_t* f_x[XCOPIES];
    auto target = [&]() {  // addresses of the item that f is in
      if (f.item == f_item) return;
      f_item = f.item;
      const auto en = entry(f.a);
      const int n0 = f.tile * OUT;
      f_valid = p.N - n0 - cr;
      f_toks = en.count;
      f_w = p.w + en.expert * p.w_estride + (int64_t)(n0 + cr) * p.ldw + cc * 16;
#pragma unroll
      for (int i = 0; i < XCOPIES; ++i) {
        if (i * TPI >= en.count) break;
        const int r = en.first + min(i * TPI + tr, en.count - 1);
        f_x[i] = p.x + (LIN ? r : l.tok[r]) * p.ldx + tc * 16;
      }
    };
    const int64_t wstep = (int64_t)RPI * p.ldw, to_up = ((int64_t)p.N - OUT) * p.ldw;
    auto fetch_w = [&](uint32_t at) {
      const bool in = f.kb * WB + cc * 16 < (I4 ? p.K / 2 : I8 ? p.K : p.K * 2);
      const int valid = in ? f_valid : -R;
      const uint8_t* src = f_w + (int64_t)f.kb * WB;
#pragma unroll
      for (int i = 0; i < R / RPI; ++i) {
        if (GU && i * RPI == OUT) src += to_up;
        // (rows 4 apart: f differs in bit 1)
        cp16((at + w_dst + i * RPI * WB) ^ (RPI == 4 && (i & 1) ? 32u : 0u), src, i * RPI % OUT < valid);
        src += wstep;
      }
    };
    auto fetch_x = [&](uint32_t at) {
      const bool in = f.kb * XB + tc * 16 < (LIN ? p.K : p.K * 2);
#pragma unroll
      for (int i = 0; i < XCOPIES; ++i) {
        if (i * TPI >= f_toks) break;
        const int m = i * TPI + tr;
        if (m < xt) cp16(at + R * WB + m * XB + xswz(tc, m) * 16, f_x[i] + f.kb * XB, in);
      }
    };

    // scales of a unit: a lane reads those of rows lane and lane + 32 of the tile
    constexpr int NS = I4 ? (FINE ? 4 : 1) : 1;
    uint16_t s_next[2][NS];  // as loaded: turning them into numbers here would wait for them
    uint8_t z_next[2][NS];
    const uint16_t* sp[2];
    const uint8_t* zp[2];
    int s_item = -1;
    auto scales = [&](const Walk& w) {
      if constexpr (I4) {
        if (w.item != s_item) {
          s_item = w.item;
          const int e = entry(w.a).expert, n0 = w.tile * OUT + lane;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t row = (int64_t)(h ? p.N : 0) + min(n0, p.N - 1);
            sp[h] = reinterpret_cast<const uint16_t*>(p.scale) + e * p.s_estride + row * p.lds;
            if (ZP) zp[h] = p.zero + e * p.z_estride + row * p.ldz;
          }
        }
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const int k = w.kb * KU + j * 32;
          const int gi = min(k, p.K - 1) >> p.group_shift;  // past the end: any finite sum of zeros
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            s_next[h][j] = k < p.K ? sp[h][gi] : (uint16_t)0;
            if (ZP) z_next[h][j] = zp[h][gi];
          }
        }
      }
    };

    Sum acc[MT][NT][4];
    float part[MT][NT][4];  // INT8: sums of the last units, exact; BF16: all sums
    int folded = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[mt][nt][i] = 0;
          part[mt][nt][i] = 0.f;
        }
    auto fold = [&]() {
      if constexpr (!I4) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if constexpr (I8)
                acc[mt][nt][i] += __float2int_rn(part[mt][nt][i]);
              else
                acc[mt][nt][i] = part[mt][nt][i];
              part[mt][nt][i] = 0.f;
            }
        folded = 0;
      }
    };

    const int pre = depth - 1;
#pragma unroll 1
    for (int d = 0; d < pre; ++d) {
      if (f.u < u1) {
        target();
        fetch_w(ring + d * stage);
        fetch_x(ring + d * stage);
      }
      cp_commit();
      f.next(W, nblk, ne);
    }

    Walk c, n;  // the unit to compute, and the one after it
    c.set(u0 + warp, nblk, ne);
    n = c;
    int done = item0, c_item = -1;
    bool mine = false;  // a unit of item `done` has been added
    float inv[NT] = {};
    uint32_t slot = 0, to_slot = pre;
    const int cap_t = xt - 1;
    if (c.u < u1) scales(c);
#pragma unroll 1
    for (;;) {
      const int to = c.u < u1 ? c.item : item1 + 1;
#pragma unroll 1
      for (; done < to; ++done) {
        // leave the sums of item `done` to the last warp
        const int b = (done - item0) % buffers;
        if (done - item0 >= buffers) bar_sync<kEmpty, THREADS>(b);
        if (mine) {
          fold();
          Sum* s = reinterpret_cast<Sum*>(smem + lay.lists + b * buffer) + warp * xt * kPitch;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (nt * 8 + 2 * t + (i & 1) < xt)
                  s[(nt * 8 + 2 * t + (i & 1)) * kPitch + mt * 16 + g + 8 * (i >> 1)] = acc[mt][nt][i];
                acc[mt][nt][i] = 0;
              }
          mine = false;
        }
        if (done < item1) bar_arrive<kFull, THREADS>(b);
      }
      if (c.u >= u1) break;
      mine = true;
      if (I8 && !LIN && c.item != c_item) {
        c_item = c.item;
        const auto en = entry(c.a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          inv[nt] = s_inv[l.tok[en.first + min(nt * 8 + g, en.count - 1)]];
        }
      }
      cp_wait(pre - 1);
      __syncwarp();  // every lane's copies of this unit have landed, and the unit before is read
      if (f.u < u1) {
        target();
        fetch_w(ring + to_slot * stage);
        fetch_x(ring + to_slot * stage);
      }
      cp_commit();
      f.next(W, nblk, ne);
      if (++to_slot == (uint32_t)depth) to_slot = 0;
      const uint32_t wat = ring + slot * stage + g * WB, xat = ring + slot * stage + R * WB;
      if (++slot == (uint32_t)depth) slot = 0;
      uint32_t sz[2][NS];  // a scale leaves the low bits of its fp32 image free for the zero point
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < NS; ++j) sz[h][j] = I4 ? (uint32_t)s_next[h][j] << 16 | (ZP ? z_next[h][j] : 0u) : 0u;
      n.next(W, nblk, ne);
      if (n.u < u1) scales(n);

      if constexpr (I4) {
        uint32_t wv[MT][2][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = wat + (mt * 16 + h * 8) * WB;
            if constexpr (FINE) {
              // word t of every 32-k piece, so that an MMA stays inside one group
#pragma unroll
              for (int j = 0; j < 4; ++j) wv[mt][h][j] = lds4(at + (j ^ swz(g)) * 16 + t * 4);
            } else {
              const uint4 v = lds16(at + (t ^ swz(g)) * 16);
              wv[mt][h][0] = v.x;
              wv[mt][h][1] = v.y;
              wv[mt][h][2] = v.z;
              wv[mt][h][3] = v.w;
            }
          }
        uint32_t negz[MT][2];
        float sc[MT][2], grp[MT][NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j == 0 || FINE) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t v = __shfl_sync(0xffffffffu, sz[mt / 2][FINE ? j : 0], mt % 2 * 16 + h * 8 + g);
                sc[mt][h] = 64.f * (p.scale_fp16 ? __half2float(__ushort_as_half(v >> 16)) : __uint_as_float(v & 0xFFFF0000u));
                // -z / 64 from z's pattern: z 2^-133 times -2^127
                negz[mt][h] = ZP ? fma_bf16x2(__byte_perm(v, 0u, 0x4040), 0xFF00FF00u, 0u) : 0xBE00BE00u;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) grp[mt][nt][2 * h] = grp[mt][nt][2 * h + 1] = 0.f;
              }
          }
          uint4 bx[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int m = min(nt * 8 + g, cap_t);
            bx[nt] = pair_up(lds16(xat + m * XB + xswz(FINE ? j * 4 + t : t * 4 + j, m) * 16));
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t q0[4], q1[4];
            codes_to_bf16(wv[mt][0][j], negz[mt][0], q0);
            codes_to_bf16(wv[mt][1][j], negz[mt][1], q1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_bf16_16816(grp[mt][nt], q0[0], q1[0], q0[1], q1[1], bx[nt].x, bx[nt].y);
              mma_bf16_16816(grp[mt][nt], q0[2], q1[2], q0[3], q1[3], bx[nt].z, bx[nt].w);
            }
          }
          if (FINE || j == 3) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][nt][i] = fmaf(sc[mt][i >> 1], grp[mt][nt][i], acc[mt][nt][i]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint4 wv[MT][2];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) wv[mt][h] = lds16(wat + (mt * 16 + h * 8) * WB + ((4 * j + t) ^ swz(g)) * 16);
          if constexpr (I8) {
            uint32_t b[NT][8];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int m = min(nt * 8 + g, cap_t);
              if constexpr (LIN) {
                const uint4 v = lds16(xat + m * XB + xswz(4 * j + t, m) * 16);
                s8x4_to_f16x2x2(v.x, b[nt][0], b[nt][1]);
                s8x4_to_f16x2x2(v.y, b[nt][2], b[nt][3]);
                s8x4_to_f16x2x2(v.z, b[nt][4], b[nt][5]);
                s8x4_to_f16x2x2(v.w, b[nt][6], b[nt][7]);
              } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint4 v = lds16(xat + m * XB + xswz(8 * j + 2 * t + i, m) * 16);
                  b[nt][4 * i] = quant2(v.x, inv[nt]);
                  b[nt][4 * i + 1] = quant2(v.y, inv[nt]);
                  b[nt][4 * i + 2] = quant2(v.z, inv[nt]);
                  b[nt][4 * i + 3] = quant2(v.w, inv[nt]);
                }
              }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              const uint32_t lo[4] = {wv[mt][0].x, wv[mt][0].y, wv[mt][0].z, wv[mt][0].w};
              const uint32_t hi[4] = {wv[mt][1].x, wv[mt][1].y, wv[mt][1].z, wv[mt][1].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t a0, a1, a2, a3;
                s8x4_to_f16x2x2(lo[i], a0, a2);
                s8x4_to_f16x2x2(hi[i], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16_16816(part[mt][nt], a0, a1, a2, a3, b[nt][2 * i], b[nt][2 * i + 1]);
              }
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int m = min(nt * 8 + g, cap_t);
              const uint4 v = lds16(xat + m * XB + xswz(4 * j + t, m) * 16);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma_bf16_16816(part[mt][nt], wv[mt][0].x, wv[mt][1].x, wv[mt][0].y, wv[mt][1].y, v.x, v.y);
                mma_bf16_16816(part[mt][nt], wv[mt][0].z, wv[mt][1].z, wv[mt][0].w, wv[mt][1].w, v.z, v.w);
              }
            }
          }
        }
        if (I8 && ++folded == 8) fold();  // 1024 k: sums of at most 2^24
      }
      c = n;
    }
  }

  // ------------------------------------------------------------------ sums and results: rows lane, lane + 32
  // 0: the part of an item that began in an earlier CTA, 1: of one that ends in a later CTA
  auto slot_of = [&](int cta, int tail) {
    return reinterpret_cast<Sum*>(p.slots + ((int64_t)cta * 2 + tail) * (TT * R)) + lane;
  };
  struct Item {
    int it, units, w0, n;  // its units here, the warp that has the first; row of a lane
    const Sum* sums;
    bool cut;
    float ws[2], bias[2];
  };
  auto item_of = [&](int it, const Walk& c, int expert) {
    Item m;
    const int ua = max(u0, it * nblk);
    m.it = it;
    m.units = min(min(u1, (it + 1) * nblk) - ua, W);
    m.w0 = (ua - u0) % W;
    m.sums = reinterpret_cast<const Sum*>(smem + lay.lists + (it - item0) % buffers * buffer) + lane;
    m.cut = it * nblk < u0 || (it + 1) * nblk > u1;
    m.n = c.tile * OUT + lane;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m.ws[h] = 1.f;
      m.bias[h] = 0.f;
      const int row = GU ? m.n : m.n + 32 * h;
      if (row < p.N) {
        if (I8)
          m.ws[h] = reinterpret_cast<const float*>(p.scale)[LIN ? (p.lds ? row : 0)
                                                                : expert * p.s_estride + (GU && h ? p.N : 0) + row];
        if (LIN && p.bias) m.bias[h] = bf16_bits_to_f32(p.bias[row]);
      }
    }
    return m;
  };
  auto own = [&](const Item& m, int k, Sum (&v)[2]) {  // the sums of this CTA's warps
    v[0] = v[1] = 0;
    int w = m.w0;
#pragma unroll 4
    for (int i = 0; i < m.units; ++i) {
      const Sum* q = m.sums + (w * xt + k) * kPitch;
      v[0] += q[0];
      v[1] += q[32];
      if (++w == W) w = 0;
    }
  };
  auto leave = [&](const Item& m, int k) {
    Sum v[2], *to = slot_of(blockIdx.x, m.it * nblk >= u0) + k * R;
    own(m, k, v);
    __stcg(to, v[0]);
    __stcg(to + 32, v[1]);
  };
  // by one thread: counts a part of item `it` in; true for the last one, which finds all parts stored
  auto last_part = [&](int it) {
    const int c0 = it * nblk / share, c1 = ((it + 1) * nblk - 1) / share;
    const unsigned before = atomicAdd(p.tickets + c0, 1u);
    if (before == (unsigned)(c1 - c0)) p.tickets[c0] = 0u;
    return before == (unsigned)(c1 - c0);
  };
  auto joined = [&](const Item& m, int k, Sum (&v)[2]) {  // all parts in the order of K
    const int c0 = m.it * nblk / share, c1 = ((m.it + 1) * nblk - 1) / share;
    v[0] = v[1] = 0;
#pragma unroll 4
    for (int q = c0; q <= c1; ++q) {
      const Sum* from = slot_of(q, q == c0) + k * R;
      v[0] += __ldcg(from);
      v[1] += __ldcg(from + 32);
    }
  };
  auto result = [&](const Item& m, int place, const Sum (&v)[2]) {  // of pair or token `place`
    float f[2] = {(float)v[0], (float)v[1]};
    if constexpr (GU) {
      const int pair = l.pair[place];
      if constexpr (I8) {
        const float xs = s_xs[l.tok[place]];
        f[0] = f[0] * xs * m.ws[0];
        f[1] = f[1] * xs * m.ws[1];
      }
      const uint16_t hb = f32_to_bf16_rn(gated_act(f[0], f[1], p.alpha, p.limit));
      if (m.n < p.N) p.h[pair * p.ldh + m.n] = hb;
      if (I8) {
        const unsigned top = __reduce_max_sync(0xffffffffu, m.n < p.N ? (unsigned)(hb & 0x7FFF) << 16 : 0u);
        if (lane == 0) atomicMax(p.amax + pair, top);
      }
    } else {
      const float xs = p.x_scale[place];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (m.n + 32 * h >= p.N) continue;
        const float o32 = __fmul_rn(__fmul_rn(f[h], xs), m.ws[h]);
        const int64_t at = (int64_t)place * p.ldy + m.n + 32 * h;
        if (p.out_type == QL_OUT_FP32) {
          reinterpret_cast<float*>(p.y)[at] = p.bias ? o32 + m.bias[h] : o32;
        } else if (p.out_type == QL_OUT_FP16) {
          __half o = __float2half_rn(o32);
          if (p.bias) o = __float2half_rn(__half2float(o) + m.bias[h]);
          reinterpret_cast<__half*>(p.y)[at] = o;
        } else {
          uint16_t o = f32_to_bf16_rn(o32);
          if (p.bias) o = f32_to_bf16_rn(bf16_bits_to_f32(o) + m.bias[h]);
          reinterpret_cast<uint16_t*>(p.y)[at] = o;
        }
      }
    }
  };

  // All items but the last by the last warp, while the others go on.  Only the first can be shared with other
  // CTAs; it is joined at the end, by all warps
  __shared__ bool s_join[2];  // this CTA has the last part of its first, its last item
  if (warp == W) {
    if (lane == 0) s_join[0] = false;
    Walk c;
    c.set(item0 * nblk, nblk, ne);
#pragma unroll 1
    for (int it = item0; it < item1; ++it) {
      const auto en = entry(c.a);
      const int b = (it - item0) % buffers;
      const Item m = item_of(it, c, en.expert);
      bar_sync<kFull, THREADS>(b);
#pragma unroll 1
      for (int k = 0; k < en.count; ++k) {
        if (m.cut) {
          leave(m, k);
          continue;
        }
        Sum v[2];
        own(m, k, v);
        result(m, en.first + k, v);
      }
      __syncwarp();
      if (it + buffers <= item1) bar_arrive<kEmpty, THREADS>(b);
      if (m.cut) {
        __threadfence();
        __syncwarp();
        if (lane == 0) s_join[0] = last_part(it);
      }
      c.next(nblk, nblk, ne);
    }
  }
  __syncthreads();
  // the last item by all warps, a token each
  Walk c;
  c.set(item1 * nblk, nblk, ne);
  const auto en = entry(c.a);
  const Item m = item_of(item1, c, en.expert);
  if (m.cut) {
#pragma unroll 1
    for (int k = warp; k < en.count; k += W + 1) leave(m, k);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) s_join[1] = last_part(item1);
    __syncthreads();
  } else {
#pragma unroll 1
    for (int k = warp; k < en.count; k += W + 1) {
      Sum v[2];
      own(m, k, v);
      result(m, en.first + k, v);
    }
  }
  __threadfence();  // the other parts were fenced before their counts
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (which ? !m.cut || !s_join[1] : !s_join[0]) continue;
    const int it = which ? item1 : item0;
    c.set(it * nblk, nblk, ne);
    const auto of = entry(c.a);
    const Item j = item_of(it, c, of.expert);
#pragma unroll 1
    for (int k = warp; k < of.count; k += W + 1) {
      Sum v[2];
      joined(j, k, v);
      result(j, of.first + k, v);
    }
  }
}

template <int FMT, int MODE, int NT, bool FINE, bool ZP>
cudaError_t launch(const StreamArgs& a, cudaStream_t st) {
  constexpr int W = compute_warps(FMT);
  auto* kfn = stream_kernel<FMT, MODE, NT, FINE, ZP>;
  static OncePerDevice once;
  if (const cudaError_t e = raise_smem_limit(kfn, once); e != cudaSuccess) return e;
  const int P = MODE == STREAM_LINEAR ? 0 : a.M * a.topk;
  const Layout l = {list_bytes(FMT, P), kSmem};
  static_assert(ring_stages(FMT, MODE, MODE == STREAM_LINEAR ? 0 : kMoeMaxTokens * kMoeMaxTopk, NT * 8) >= 2,
                "two stages with the most pairs, and the most tokens of an entry");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kNumSMs, 1, 1);
  cfg.blockDim = dim3((W + 1) * 32, 1, 1);
  cfg.dynamicSmemBytes = (size_t)l.total;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, a, l);
}

}  // namespace

size_t stream_slot_bytes(int64_t M) {
  const int64_t columns = M < kLinearTokens ? kLinearTokens : M;
  return (size_t)kNumSMs * 2 * columns * R * 4;
}

cudaError_t launch_gate_up(int fmt, const StreamArgs& a, cudaStream_t st) {
  constexpr int GU = STREAM_GATE_UP;
  if (fmt == STREAM_BF16) return launch<STREAM_BF16, GU, 1, false, false>(a, st);
  if (fmt == STREAM_INT8) return launch<STREAM_INT8, GU, 1, false, false>(a, st);
  if (a.group_shift < 7)
    return a.zero ? launch<STREAM_INT4, GU, 1, true, true>(a, st) : launch<STREAM_INT4, GU, 1, true, false>(a, st);
  return a.zero ? launch<STREAM_INT4, GU, 1, false, true>(a, st) : launch<STREAM_INT4, GU, 1, false, false>(a, st);
}

cudaError_t launch_linear(const StreamArgs& a, cudaStream_t st) {
  if (a.M <= 8) return launch<STREAM_INT8, STREAM_LINEAR, 1, false, false>(a, st);
  return launch<STREAM_INT8, STREAM_LINEAR, 2, false, false>(a, st);
}

}  // namespace ql
