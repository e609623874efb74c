// The gated feed-forward block for more than a few tokens, and its backward pass, on the
// 5th-generation tensor cores.
//
//   forward   g = x Wg^T, u = x Wu^T   (W13 = [Wg; Wu], rows [0, I) gate and [I, 2I) up)
//             h = bf16( silu(a min(g, L)) * clamp(u, -L, L) )
//             checkpoint of g and u: bf16, or int8 codes with one scale per token and 128 columns
//   backward  du = dh silu(a gc) [|u| <= L],  dg = dh uc a silu'(a gc) [g <= L]
//             dx = [dg du] W13,   dW13 = [dg du]^T x
//             with gc = min(g, L), uc = clamp(u, -L, L), silu'(t) = s(t) (1 + t (1 - s(t)))
//
// One GEMM kernel, C = A B^T with bf16 operands and fp32 sums in tensor memory, in three forms:
//   FWD: A = x, B = W13 (both K-major); a tile is 256 tokens x 128 outputs, i.e. 128 gate and 128
//        up columns, so that the activation and the product run in the epilogue and g, u never
//        reach memory (but for the checkpoint)
//   DX : A = [dg du] (K-major), B = W13^T (N-major: H is contiguous), a tile is 256 x 256
//   DW : A = [dg du]^T (M-major), B = x^T (N-major), a tile is 256 x 256
// A pair of CTAs on two SMs shares a tile (cta_group::2): each holds 128 rows of A, half of B's
// 256 columns and 128 rows of the accumulator, so that an SM loads half of B.  The grid is one
// pair per two SMs; pairs take tiles in turn.  Roles in a CTA:
//   warp 0: TMA producer;  warp 1: MMA issue (first CTA of the pair only);  warp 2: tensor memory;
//   warps 4..7: epilogue, one row of the accumulator per thread.
// Two accumulators of 256 columns take turns, so a tile's epilogue runs under the next tile's
// MMAs.  Every wait is bounded; one that runs out raises QL_DEV_TIMEOUT in the status word and the
// pair leaves its loops, waits for copies and MMAs in flight and frees its tensor memory.
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdio>
#include <mutex>

#include "common.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace ql {
namespace tc {

namespace {

enum { FWD = 0, DX = 1, DW = 2 };

constexpr int kThreads = 256;
constexpr int kBlockK = 64;  // one 128-byte swizzled row of bf16
constexpr int kStages = 6;
constexpr uint32_t kHalfBytes = 128 * kBlockK * 2;  // one operand's half tile of a stage
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kDrainLimit = 1u << 22;
constexpr int kGroupM = 16;  // tile rows that run before the next tile column

struct Params {
  int rows, cols, K;        // of C; FWD: cols = I (outputs)
  int tiles_m, tiles_n, nk;
  uint16_t* out;            // bf16 [rows, ld_out]
  int64_t ld_out;
  float alpha, limit;       // FWD
  int save;                 // FWD: QL_SAVE_*
  int I;                    // FWD: row of W13 where the up rows start
  void* ckpt;               // FWD
  float* ckpt_scale;
  uint32_t* status;
  uint32_t wait_limit;
};

// ------------------------------------------------------------------ pair-of-CTAs PTX
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t in_cta(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t cluster_addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
// acquires at cluster scope: arrivals come from both CTAs
__device__ __forceinline__ bool wait2(uint64_t* bar, uint32_t parity, uint32_t limit, volatile int* abort) {
  for (uint32_t n = 0;; ++n) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if (n >= limit || (abort && *abort)) return false;
  }
}
// the box goes to this CTA's shared memory, its bytes to the barrier at cluster address `bar`
__device__ __forceinline__ void load_pair(uint32_t smem_dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// arrives on the barrier at this offset in both CTAs once the MMAs issued so far have finished
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// Matrix descriptor of an MN-major operand written by TMA with 128-byte swizzling: chunks of 64
// columns (128 bytes) x 64 k rows; leading byte offset = the next chunk of columns (8 KB),
// stride byte offset = the next 8 k rows (1 KB).
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | (uint64_t)(8192 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// kind::f16, bf16 operands (format 1), fp32 accumulator, M = 256 over the pair, N = 256; bits 15
// and 16: A / B are MN-major
constexpr uint32_t idesc_pair(bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((256u >> 3) << 17) | ((256u >> 4) << 24);
}

// tile index -> (m, n): blocks of kGroupM tile rows, the rows of a block first
__device__ __forceinline__ void tile_at(const Params& p, int t, int& m, int& n) {
  const int block = t / (kGroupM * p.tiles_n), in = t - block * kGroupM * p.tiles_n;
  const int rows = min(kGroupM, p.tiles_m - block * kGroupM);
  m = block * kGroupM + in % rows;
  n = in / rows;
}

__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ Params p) {
  constexpr bool A_MN = MODE == DW, B_MN = MODE != FWD;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_issued;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  // the stages start at the same offset in both CTAs
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = p.tiles_m * p.tiles_n;
  const uint32_t lim = p.wait_limit;
  volatile int* abort = &s_abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 8);  // four epilogue warps in each CTA
    }
    mbar_init(&done, 1);
    fence_mbar_init();
    s_abort = 0;
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  auto fail = [&]() {
    atomicOr(p.status, (uint32_t)QL_DEV_TIMEOUT);
    *abort = 1;
    st_remote(in_cta(smem_u32(&s_abort), rank ^ 1), 1);
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------- producer
      int s = 0, issued = 0;
      uint32_t ph = 1;  // the first pass over the stages finds them empty
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        int tm, tn;
        tile_at(p, t, tm, tn);
        const int ra = tm * 256 + (int)rank * 128;
        const int rb = MODE == FWD ? tn * 128 + (int)rank * p.I : tn * 256 + (int)rank * 128;
        for (int kt = 0; kt < p.nk; ++kt) {
          if (!wait2(&empty[s], ph, lim, abort)) {
            fail();
            ok = false;
            break;
          }
          const uint32_t bar = in_cta(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
          const uint32_t sa = base + (uint32_t)s * kStageBytes, sb = sa + kHalfBytes;
          const int k = kt * kBlockK;
          if (A_MN) {
            load_pair(sa, &tmA, ra, k, bar);
            load_pair(sa + 8192, &tmA, ra + 64, k, bar);
          } else {
            load_pair(sa, &tmA, k, ra, bar);
          }
          if (B_MN) {
            load_pair(sb, &tmB, rb, k, bar);
            load_pair(sb + 8192, &tmB, rb + 64, k, bar);
          } else {
            load_pair(sb, &tmB, k, rb, bar);
          }
          ++issued;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // the last stages' releases, multicast by the other CTA, land before this CTA may leave
      for (int i = 0; i < kStages && ok; ++i) {
        ok = wait2(&empty[s], ph, lim, abort);
        if (!ok) fail();
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (ok && !wait2(&done, 0, lim, abort)) fail();
      s_issued = issued;
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---------------------------------------------------------- MMA issue
      constexpr uint32_t idesc = idesc_pair(A_MN, B_MN);
      constexpr uint64_t a_step = A_MN ? 2048 / 16 : 2, b_step = B_MN ? 2048 / 16 : 2;  // 16 k
      const uint64_t a0 = A_MN ? desc_mn(base) : smem_desc_sw128(base);
      const uint64_t b0 = B_MN ? desc_mn(base + kHalfBytes) : smem_desc_sw128(base + kHalfBytes);
      int s = 0, n = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, ++n) {
        const int buf = n & 1;
        if (!wait2(&tempty[buf], (uint32_t)((n >> 1) & 1) ^ 1, lim, abort)) {
          fail();
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)buf * 256;
        for (int kt = 0; kt < p.nk; ++kt) {
          if (!wait2(&full[s], ph, lim, abort)) {
            fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = (uint64_t)s * (kStageBytes >> 4);
#pragma unroll
          for (int j = 0; j < kBlockK / 16; ++j)
            mma_pair(d, a0 + off + j * a_step, b0 + off + j * b_step, idesc, (kt | j) != 0);
          commit_pair(&empty[s]);
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (ok) commit_pair(&tfull[buf]);
      }
      commit_pair(&done);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    int n = 0;
    for (int t = pair; t < tiles; t += pairs, ++n) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int buf = n & 1;
      int got = 0;
      if (lane == 0) got = wait2(&tfull[buf], (uint32_t)(n >> 1) & 1, lim, abort);
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) {
        if (lane == 0) fail();
        break;
      }
      tc_fence_after();
      const int row = tm * 256 + (int)rank * 128 + 32 * q + lane;
      const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)buf * 256;
      if constexpr (MODE == FWD) {
        const int i0 = tn * 128;
        float inv_g = 0.f, inv_u = 0.f;
        const int64_t ipad = ckpt_pad(p.I);
        if (p.save == QL_SAVE_INT8) {
          // first pass over the accumulator: the largest |g| and |u| of the row's 128 columns
          float ag = 0.f, au = 0.f;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t rg[32], ru[32];
            tmem_ld_x32(acc + c, rg);
            tmem_ld_x32(acc + 128 + c, ru);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i0 + c + (i & ~7) < p.cols) {
                ag = max_nan(ag, fabsf(__uint_as_float(rg[i])));
                au = max_nan(au, fabsf(__uint_as_float(ru[i])));
              }
          }
          if (row < p.rows) {
            float* s = p.ckpt_scale + (int64_t)row * 2 * (ipad / 128) + tn;
            s[0] = ckpt_scale(ag, inv_g);
            s[ipad / 128] = ckpt_scale(au, inv_u);
          }
        }
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          uint32_t rg[32], ru[32];
          tmem_ld_x32(acc + c, rg);
          tmem_ld_x32(acc + 128 + c, ru);
          tmem_wait_ld();
          if (row < p.rows) {
#pragma unroll
            for (int v = 0; v < 32; v += 8) {
              const int i = i0 + c + v;
              if (i < p.cols) {
                float h[8], g[8], u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  g[j] = __uint_as_float(rg[v + j]);
                  u[j] = __uint_as_float(ru[v + j]);
                  h[j] = gated_act(g[j], u[j], p.alpha, p.limit);
                }
                store8(p.out + (int64_t)row * p.ld_out + i, h);
                if (p.save == QL_SAVE_BF16) {
                  uint16_t* ck = reinterpret_cast<uint16_t*>(p.ckpt) + (int64_t)row * 2 * ipad + i;
                  store8(ck, g);
                  store8(ck + ipad, u);
                } else if (p.save == QL_SAVE_INT8) {
                  int8_t* ck = reinterpret_cast<int8_t*>(p.ckpt) + (int64_t)row * 2 * ipad + i;
                  *reinterpret_cast<uint2*>(ck) = ckpt_codes8(g, inv_g);
                  *reinterpret_cast<uint2*>(ck + ipad) = ckpt_codes8(u, inv_u);
                }
              }
            }
          }
        }
      } else {
        const int c0 = tn * 256;
#pragma unroll 1
        for (int c = 0; c < 256; c += 32) {
          uint32_t r[32];
          tmem_ld_x32(acc + c, r);
          tmem_wait_ld();
          if (row < p.rows) {
#pragma unroll
            for (int v = 0; v < 32; v += 8) {
              if (c0 + c + v < p.cols) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(r[v + j]);
                store8(p.out + (int64_t)row * p.ld_out + c0 + c + v, f);
              }
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_remote(in_cta(smem_u32(&tempty[buf]), 0));
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (*abort) {  // set in both CTAs or in neither
    // no copy may land after the pair has left.  The stages' bytes are counted by the first CTA's
    // barriers: for a use of a stage that only one CTA got to, the other half's arrival or bytes
    // are supplied here, and the last use of every stage is waited for
    if (threadIdx.x == 0) wait2(&done, 0, kDrainLimit, nullptr);  // no MMA is reading them
    if (rank == 0 && threadIdx.x == 0) {
      int other;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other) : "r"(in_cta(smem_u32(&s_issued), 1)) : "memory");
      const int mine = s_issued, last = mine > other ? mine : other;
      for (int i = last > kStages ? last - kStages : 0; i < last; ++i) {
        uint64_t* bar = &full[i % kStages];
        if (i >= mine)
          mbar_arrive_expect_tx(bar, kStageBytes);
        else if (i >= other)
          asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                       "r"(kStageBytes)
                       : "memory");
        wait2(bar, (uint32_t)(i / kStages) & 1, kDrainLimit, nullptr);
      }
    }
    __syncthreads();
    cluster_sync_all();
  }
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ------------------------------------------------------------------ gradients of g and u
// dgu[m, i] = dg, dgu[m, I + i] = du from dh and the checkpoint, eight columns per thread.  One
// pass over memory: reads dh and the checkpoint, writes 4 bytes per output.
template <bool INT8>
__global__ void __launch_bounds__(256) gated_grad_kernel(const uint16_t* __restrict__ dh, int64_t ld_dh, int64_t M,
                                                         int I, const void* __restrict__ ckpt,
                                                         const float* __restrict__ scale, float alpha, float limit,
                                                         uint16_t* __restrict__ dgu) {
  const int64_t ipad = ckpt_pad(I);
  const int i = (blockIdx.x * 256 + threadIdx.x) * 8;
  if (i >= I) return;
  for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
    const uint4 d = *reinterpret_cast<const uint4*>(dh + m * ld_dh + i);
    float g[8], u[8];
    if constexpr (INT8) {
      const int8_t* ck = reinterpret_cast<const int8_t*>(ckpt) + m * 2 * ipad + i;
      const float* s = scale + m * 2 * (ipad / 128) + (i >> 7);
      ckpt_values8(*reinterpret_cast<const uint2*>(ck), s[0], g);
      ckpt_values8(*reinterpret_cast<const uint2*>(ck + ipad), s[ipad / 128], u);
    } else {
      const uint16_t* ck = reinterpret_cast<const uint16_t*>(ckpt) + m * 2 * ipad + i;
      bf16_values8(*reinterpret_cast<const uint4*>(ck), g);
      bf16_values8(*reinterpret_cast<const uint4*>(ck + ipad), u);
    }
    float dv[8], dg[8], du[8];
    bf16_values8(d, dv);
#pragma unroll
    for (int j = 0; j < 8; ++j) gated_grad(dv[j], g[j], u[j], alpha, limit, dg[j], du[j]);
    store8(dgu + m * 2 * I + i, dg);
    store8(dgu + m * 2 * I + I + i, du);
  }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* q = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(q);
  });
  return fn;
}

// bf16 [outer, inner], boxes of 64 columns (one swizzled 128-byte row) x box_rows
bool bf16_map(CUtensorMap* m, const void* base, int64_t inner, int64_t outer, int64_t ld, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) fprintf(stderr, "qlinear: cuTensorMapEncodeTiled failed (%d)\n", (int)r);
  return r == CUDA_SUCCESS;
}

template <int MODE>
cudaError_t run(const CUtensorMap& ta, const CUtensorMap& tb, Params& p, cudaStream_t st) {
  p.tiles_m = (p.rows + 255) / 256;
  p.tiles_n = MODE == FWD ? (p.cols + 127) / 128 : (p.cols + 255) / 256;
  p.nk = (p.K + kBlockK - 1) / kBlockK;
  static std::atomic<int> attr{0};
  if (!attr.load()) {
    const cudaError_t e = raise_smem_limit(ffn_gemm_kernel<MODE>);
    if (e != cudaSuccess) return e;
    attr.store(1);
  }
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  const int pairs = (int)(tiles < kNumSMs / 2 ? tiles : kNumSMs / 2);
  ffn_gemm_kernel<MODE><<<2 * pairs, kThreads, 1024 + kStages * kStageBytes, st>>>(ta, tb, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ffn_forward(const FfnForward& f, cudaStream_t st) {
  CUtensorMap ta, tb;
  if (!bf16_map(&ta, f.x, f.H, f.M, f.ldx, 128) || !bf16_map(&tb, f.w13, f.H, 2 * f.I, f.ldw, 128))
    return cudaErrorInvalidValue;
  Params p = {};
  p.rows = (int)f.M;
  p.cols = (int)f.I;
  p.K = (int)f.H;
  p.out = f.h;
  p.ld_out = f.ldh;
  p.alpha = f.alpha;
  p.limit = f.limit;
  p.save = f.save;
  p.I = (int)f.I;
  p.ckpt = f.ckpt;
  p.ckpt_scale = f.ckpt_scale;
  p.status = f.status;
  p.wait_limit = f.wait_limit;
  return run<FWD>(ta, tb, p, st);
}

cudaError_t launch_ffn_backward(const FfnBackward& b, cudaStream_t st) {
  const dim3 grid((unsigned)((b.I + 2047) / 2048), (unsigned)(b.M < 32768 ? b.M : 32768));
  if (b.save == QL_SAVE_INT8)
    gated_grad_kernel<true><<<grid, 256, 0, st>>>(b.dh, b.ld_dh, b.M, (int)b.I, b.ckpt, b.ckpt_scale, b.alpha, b.limit,
                                                  b.dgu);
  else
    gated_grad_kernel<false><<<grid, 256, 0, st>>>(b.dh, b.ld_dh, b.M, (int)b.I, b.ckpt, nullptr, b.alpha, b.limit,
                                                   b.dgu);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  CUtensorMap ta, tb;
  Params p = {};
  p.status = b.status;
  p.wait_limit = b.wait_limit;
  if (b.dx) {
    if (!bf16_map(&ta, b.dgu, 2 * b.I, b.M, 2 * b.I, 128) || !bf16_map(&tb, b.w13, b.H, 2 * b.I, b.ldw, 64))
      return cudaErrorInvalidValue;
    p.rows = (int)b.M;
    p.cols = (int)b.H;
    p.K = (int)(2 * b.I);
    p.out = b.dx;
    p.ld_out = b.ld_dx;
    e = run<DX>(ta, tb, p, st);
    if (e != cudaSuccess) return e;
  }
  if (b.dw13) {
    if (!bf16_map(&ta, b.dgu, 2 * b.I, b.M, 2 * b.I, 64) || !bf16_map(&tb, b.x, b.H, b.M, b.ldx, 64))
      return cudaErrorInvalidValue;
    p.rows = (int)(2 * b.I);
    p.cols = (int)b.H;
    p.K = (int)b.M;
    p.out = b.dw13;
    p.ld_out = b.ld_dw;
    e = run<DW>(ta, tb, p, st);
  }
  return e;
}

}  // namespace tc
}  // namespace ql
