// y = (acc x_scale) w_scale, acc = x_q w^T on 8-bit codes, for more than a few tokens, on the
// 5th-generation tensor cores.
//
// sm_103a has no integer tcgen05 product.  Codes are exact in f16 and a product of two is exact in
// fp32, so the sums run as kind::f16 with fp32 accumulators: 1024 k add at most 1024 * 128 * 128 =
// 2^24 to an output, up to which fp32 holds every whole number, so accumulators are moved to int32
// registers every 1024 k.  acc is exact for any codes.
//
// A tile is 256 weight rows (the products' M) by `width` tokens, shared by a pair of CTAs on two SMs
// (cta_group::2): each holds 128 rows of weights, half of the tokens and 128 rows of the accumulator.
// The weights stay 8-bit up to the SM: converter warps widen them into tensor memory, which holds the
// products' A operand, so their f16 form costs shared memory no bandwidth.  Tokens are widened once,
// by a launch before (their f16 form is read by every row of tiles).  Roles in a CTA:
//   warp 0: TMA producer;  warp 1: MMA issue, warp 3: tokens' arrival (both in the first CTA of the pair
//   only);  warp 2: tensor memory;
//   warps 4..11: accumulators to int32 registers (a row and half of the columns per thread), results;
//   warps 12..19: weights to f16 (a row and half of a stage's 128 k per thread).
// Two accumulators take turns every 1024 k, three A buffers every 128 k: 2 * 160 + 3 * 64 columns.
// Pairs take whole tiles in turn.  What is left over, less than one tile each, is cut into equal
// stretches of 128-k stages; a pair leaves the sums of its part of a tile in a slot of the workspace and
// counts in on the tile's ticket, and the one that completes the count adds the parts (whole numbers:
// in any order).  Nobody waits for another pair.
// Bound by a stage's chain of barriers (tokens and weights loaded, widened, multiplied, freed): 0.5 us
// for 128 k where the products alone take 0.35 (640 clocks); the pipe is busy two thirds of the time.
// 4096x17408x5120 480 us (1.52 PFLOP/s), 777x10240x5120 66 us, 19x5120x17408 34 us.  On the way there,
// at 4096x17408x5120 with quantising: 907 us; 719 without cluster-wide release and acquire at every
// barrier; 517 with one wait and one commit for 128 k and barriers tested early.  Left out there: tiles of
// 192 tokens 511, of 128 tokens with 256-k stages 580, three converter groups 548, converters on
// alternating stages 573 (spills), one lane polling for its warp 837 where all lanes took 685.
// Every wait is bounded; one that runs out raises QL_DEV_TIMEOUT in the status word and the pair leaves
// its loops, waits for copies and products in flight and frees its tensor memory.  Its part of a tile
// counts in as missing, so that the next call finds the tickets as it needs them.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <cstdio>
#include <mutex>

#include "common.cuh"
#include "gemm_codes.h"
#include "internal.h"
#include "tc_pair.cuh"
#include "tc_ptx.cuh"

namespace ql {
namespace tc {

namespace {

constexpr int kThreads = 640;
constexpr int kPairs = kNumSMs / 2;
constexpr int kStageK = 128;
constexpr int kGroup = 8;  // stages of an accumulator: 1024 k
constexpr int kMaxWidth = 160;
constexpr int kStages = 5;
constexpr uint32_t kWBytes = 128 * kStageK;                     // 8-bit weights of a stage
constexpr uint32_t kXTile = kMaxWidth / 2 * 128;                // f16 tokens of 64 k
constexpr uint32_t kStageBytes = kWBytes + 2 * kXTile;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kAccCols = kMaxWidth, kACol = 2 * kAccCols, kACols = 64;
constexpr int kABufs = (kTmemCols - kACol) / kACols;  // a stage's weights each
constexpr uint32_t kDrainLimit = 1u << 22;
constexpr int kBlockRows = 16;  // tile rows that run before the next tile column
constexpr unsigned kMissing = 1u << 16;  // of a ticket: a part that was not computed
static_assert(kABufs == 3 && kABufs < kStages, "tensor memory");
// registers a thread of the five warpgroups; the launch gives each 96 (640 threads share 65536)
constexpr int kRegsIssue = 48, kRegsSums = 152, kRegsWiden = 64;
static_assert(kRegsIssue + 2 * kRegsSums + 2 * kRegsWiden <= 5 * 96, "register split");

struct Params {
  int M, N, nk, width;
  int tiles_n, tiles_m;  // of weight rows, of tokens
  int whole;             // tiles taken whole, pair after pair
  int share;             // stages of the rest for each pair
  int rest;              // tiles of the rest
  int32_t* slots;        // [pairs][2 parts][2 CTAs][width][128]
  unsigned* tickets;     // [rest][2 CTAs], zero between calls
  const float* x_scale;
  const float* w_scale;
  int w_scale_len;
  const uint16_t* bias;
  void* y;
  int64_t ldy;
  int out_type;
  uint32_t* status;
  uint32_t wait_limit;
};

// what a pair works on, one item after the other: whole tiles, then its stretch of the rest
struct Walk {
  int t, pair, u, end;
  __device__ Walk(const Params& p, int pair_) : t(pair_), pair(pair_) {
    const int64_t total = (int64_t)p.rest * p.nk, a = (int64_t)pair_ * p.share;
    u = (int)(a < total ? a : total);
    end = (int)(a + p.share < total ? a + p.share : total);
  }
  __device__ bool next(const Params& p, int& tile, int& k0, int& k1) {
    if (t < p.whole) {
      tile = t;
      k0 = 0;
      k1 = p.nk;
      t += kPairs;
      return true;
    }
    if (u >= end) return false;
    const int j = u / p.nk;
    tile = p.whole + j;
    k0 = u - j * p.nk;
    k1 = min(p.nk, end - j * p.nk);
    u += k1 - k0;
    return true;
  }
};

__device__ __forceinline__ void tile_at(const Params& p, int t, int& n, int& m) {
  const int block = t / (kBlockRows * p.tiles_m), in = t - block * kBlockRows * p.tiles_m;
  const int rows = min(kBlockRows, p.tiles_n - block * kBlockRows);
  n = block * kBlockRows + in % rows;
  m = in / rows;
}

__device__ __forceinline__ void mma_pair_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st_u32x32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// What these order is tensor memory, written and read: tcgen05 fences on both sides of the barrier do
// that.  No other memory is handed over, so neither side pays for a cluster-wide release or acquire
// (with them a stage of 128 k took 1.15 us, whatever was left out of it).
__device__ __forceinline__ void arrive_tmem(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t limit, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit, abort));
}
// asked early and used later: the answer takes about 250 cycles, the phase complete or not
__device__ __forceinline__ uint32_t ask(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok;
}
// a barrier of the eight warps that hold the results; true if `bad` is true in one of their threads
__device__ __forceinline__ bool results_any(bool bad) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 256, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)bad)
      : "memory");
  return r != 0;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    codes_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  // full_w: 8-bit weights of a stage (this CTA's); full_x: both CTAs' tokens (first CTA's); ready: both
  // CTAs have widened a stage's weights, and its tokens are there (first CTA's); empty: its products
  // have finished, the stage and its A buffer are free
  __shared__ uint64_t full_w[kStages], full_x[kStages], empty[kStages], ready[kABufs], dfull[2], dempty[2], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_issued, s_ahead, s_last;
  __shared__ float s_xs[kMaxWidth];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const int pair = blockIdx.x >> 1;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;  // the same offset in both CTAs
  const int hw = p.width / 2;
  const uint32_t x_bytes = (uint32_t)hw * 128;  // of 64 k
  const uint32_t lim = p.wait_limit;
  // the results wait for a group's products, the others for a stage
  const uint32_t lim_group = (uint32_t)min((uint64_t)lim * 2, (uint64_t)0xFFFFFFFEu);
  volatile int* abort = &s_abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_w[s], 1);
      mbar_init(&full_x[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kABufs; ++b) mbar_init(&ready[b], 17);  // eight converter warps in each CTA, the first CTA's warp 3
    for (int b = 0; b < 2; ++b) {
      mbar_init(&dfull[b], 1);
      mbar_init(&dempty[b], 16);  // eight result warps in each CTA
    }
    mbar_init(&done, 1);
    fence_mbar_init();
    s_abort = 0;
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
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
  // What the launch before (codes_f16_kernel, which has waited for everything earlier) writes is the
  // tokens alone: only their loads wait for it
  pdl_launch_dependents();
  const uint32_t tmem = s_tmem;
  auto fail = [&]() {
    atomicOr(p.status, (uint32_t)QL_DEV_TIMEOUT);
    *abort = 1;
    st_remote(in_cta(smem_u32(&s_abort), rank ^ 1), 1);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue) : "memory");
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      const bool leader = elect_one();
      int s = 0, issued = 0, ahead = 0;  // ahead: stages whose weights are under way
      uint32_t ph = 1;                   // the first pass over the stages finds them empty
      bool ok = true;
      int t, k0, k1;
      auto stage_at = [&](int i) { return smem_raw + (base - smem_u32(smem_raw)) + (size_t)i * kStageBytes; };
      auto load_w = [&](int i, int kt, int rw) {
        mbar_arrive_expect_tx(&full_w[i], kWBytes);
        tma_load_2d(stage_at(i), &tmW, kt * kStageK, rw, &full_w[i]);
      };
      for (Walk w(p, pair); ahead < kStages && w.next(p, t, k0, k1);) {
        int tn, tm;
        tile_at(p, t, tn, tm);
        for (int kt = k0; kt < k1 && ahead < kStages; ++kt, ++ahead)
          if (leader) load_w(ahead, kt, tn * 256 + (int)rank * 128);
      }
      __syncwarp();
      pdl_wait();
      for (Walk w(p, pair); ok && w.next(p, t, k0, k1);) {
        int tn, tm;
        tile_at(p, t, tn, tm);
        const int rw = tn * 256 + (int)rank * 128, rx = tm * p.width + (int)rank * hw;
        for (int kt = k0; kt < k1; ++kt) {
          if (!wait_warp(&empty[s], ph, lim, abort)) {
            if (leader) fail();
            ok = false;
            break;
          }
          if (leader) {
            const uint32_t bar = in_cta(smem_u32(&full_x[s]), 0), at = smem_u32(stage_at(s));
            if (issued >= ahead) load_w(s, kt, rw);
            if (rank == 0) mbar_arrive_expect_tx(&full_x[s], 4 * x_bytes);
            load_pair(at + kWBytes, &tmX, kt * kStageK, rx, bar);
            load_pair(at + kWBytes + kXTile, &tmX, kt * kStageK + 64, rx, bar);
          }
          __syncwarp();
          ++issued;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // the last stages' releases, multicast by the other CTA, land before this CTA may leave
      for (int i = 0; i < kStages && ok; ++i) {
        ok = wait2_warp(&empty[s], ph, lim, abort);
        if (!ok && leader) fail();
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (ok && !wait2_warp(&done, 0, lim, abort) && leader) fail();
      if (leader) {
        s_issued = issued;
        s_ahead = ahead;
      }
    } else if (warp == 1 && rank == 0) {
      // ---------------------------------------------------------- MMA issue
      const bool leader = elect_one();
      // f16 operands (format 0), fp32 accumulator, M = 256 over the pair, N = width
      const uint32_t idesc = (1u << 4) | ((uint32_t)(p.width >> 3) << 17) | ((256u >> 4) << 24);
      const uint64_t x0 = smem_desc_sw128(base + kWBytes);
      int s = 0, a = 0, g = 0;  // stage, A buffer, groups so far
      uint32_t aph = 0;
      bool ok = true;
      int t, k0, k1;
      for (Walk w(p, pair); ok && w.next(p, t, k0, k1);) {
        for (int kt = k0; kt < k1; ++kt) {
          const bool first = (kt - k0) % kGroup == 0, last = (kt - k0) % kGroup == kGroup - 1 || kt == k1 - 1;
          const int buf = g & 1;
          // (a wait costs this warp 0.1 us, waited for or not: one for each 128 k, and one commit)
          if ((first && !wait_warp(&dempty[buf], (uint32_t)((g >> 1) & 1) ^ 1, lim, abort)) ||
              !wait_warp(&ready[a], aph, lim, abort)) {
            if (leader) fail();
            ok = false;
            break;
          }
          tc_fence_after();
          if (leader) {
            const uint32_t d = tmem + (uint32_t)buf * kAccCols, at = tmem + kACol + (uint32_t)a * kACols;
            const uint64_t x = x0 + (uint64_t)s * (kStageBytes >> 4);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              mma_pair_ta(d, at + j * 8, x + (j >> 2) * (kXTile >> 4) + (j & 3) * 2, idesc, !first || j != 0);
            commit_pair(&empty[s]);
            if (last) commit_pair(&dfull[buf]);
          }
          __syncwarp();
          if (last) ++g;
          if (++a == kABufs) {
            a = 0;
            aph ^= 1;
          }
          if (++s == kStages) s = 0;
        }
      }
      if (leader) commit_pair(&done);
    } else if (warp == 3 && rank == 0) {
      // ---------------------------------------------------------- a stage's tokens are there
      int s = 0, a = 0, n = 0;
      uint32_t ph = 0, aph = 1;
      int t, k0, k1;
      for (Walk w(p, pair); w.next(p, t, k0, k1);) n += k1 - k0;
      for (int i = 0; i < n; ++i) {
        // (the buffer's count for the stage before it is complete)
        if (!wait_warp(&ready[a], aph, lim, abort) || !wait_warp(&full_x[s], ph, lim, abort)) {
          if (lane == 0) fail();
          break;
        }
        if (lane == 0) mbar_arrive(&ready[a]);
        if (++a == kABufs) {
          a = 0;
          aph ^= 1;
        }
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------------------ int32 sums, results
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSums) : "memory");
    pdl_wait();  // scales are read, results written
    const int q = warp & 3, half = (warp - 4) >> 2;  // tensor-memory lane quadrant, column half
    const int r = 32 * q + lane;                     // row of this CTA's 128
    const int cols = p.width / 2;                    // of a thread
    const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * cols);
    const int tid = threadIdx.x - 128;
    auto count_in = [&](int j, unsigned add) {
      const int64_t a = (int64_t)j * p.nk;
      const unsigned parts = (unsigned)((a + p.nk - 1) / p.share - a / p.share + 1);
      unsigned* ticket = p.tickets + 2 * j + rank;
      const unsigned before = atomicAdd(ticket, add);
      if ((before & (kMissing - 1)) != parts - 1) return false;
      *ticket = 0;
      return before < kMissing;
    };
    Walk w(p, pair);
    int g = 0, t, k0, k1;
    bool ok = true;
    while (w.next(p, t, k0, k1)) {
      int tn, tm;
      tile_at(p, t, tn, tm);
      int32_t acc[kMaxWidth / 2];
#pragma unroll
      for (int i = 0; i < kMaxWidth / 2; ++i) acc[i] = 0;
      for (int k = k0; k < k1 && ok; k += kGroup, ++g) {
        const int buf = g & 1;
        int got = 0;
        if (lane == 0) got = mbar_wait(&dfull[buf], (uint32_t)(g >> 1) & 1, lim_group, abort);
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got && lane == 0) fail();
        if (!got) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < kMaxWidth / 2; c += 32)
          if (c < cols) {  // (past this half: the other's columns, not used)
            uint32_t v[32];
            tmem_ld_x32(at + (uint32_t)buf * kAccCols + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c + i < kMaxWidth / 2) acc[c + i] += __float2int_rn(__uint_as_float(v[i]));
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_tmem(in_cta(smem_u32(&dempty[buf]), 0));
      }
      if (results_any(!ok)) {  // all eight warps or none: they meet at barriers below
        ok = false;
        // a pair that gave up counts its parts in as missing
        if (tid == 0) {
          if (t >= p.whole) count_in(t - p.whole, 1u + kMissing);
          while (w.next(p, t, k0, k1))
            if (t >= p.whole) count_in(t - p.whole, 1u + kMissing);
        }
        break;
      }
      const int m0 = tm * p.width + half * cols, n = tn * 256 + (int)rank * 128 + r;
      if (k1 - k0 != p.nk) {
        const int j = t - p.whole;
        auto slot_of = [&](int64_t pr) {
          const int part = pr * p.share / p.nk == j ? 0 : 1;
          return p.slots + (((pr * 2 + part) * 2 + rank) * p.width + half * cols) * 128 + r;
        };
        int32_t* mine = slot_of(pair);
#pragma unroll
        for (int c = 0; c < kMaxWidth / 2; ++c)
          if (c < cols) __stcg(mine + c * 128, acc[c]);
        __threadfence();
        results_any(false);  // every warp's part is stored and fenced
        if (tid == 0) s_last = count_in(j, 1u);
        results_any(false);
        if (!s_last) continue;
        __threadfence();  // the other parts were fenced before their counts
        const int64_t a = (int64_t)j * p.nk;
        for (int64_t pr = a / p.share; pr <= (a + p.nk - 1) / p.share; ++pr) {
          if (pr == pair) continue;
          const int32_t* from = slot_of(pr);
#pragma unroll
          for (int c0 = 0; c0 < kMaxWidth / 2; c0 += 16)
            if (c0 < cols) {
              int32_t v[16];
#pragma unroll
              for (int c = 0; c < 16; ++c) v[c] = __ldcg(from + (c0 + c) * 128);
#pragma unroll
              for (int c = 0; c < 16; ++c) acc[c0 + c] += v[c];
            }
        }
      }
      for (int i = tid; i < p.width; i += 256) s_xs[i] = tm * p.width + i < p.M ? p.x_scale[tm * p.width + i] : 0.f;
      results_any(false);
      if (n < p.N) {
        const float ws = p.w_scale[p.w_scale_len > 1 ? n : 0];
        const float bias = p.bias ? bf16_bits_to_f32(p.bias[n]) : 0.f;
        const int rows = min(cols, p.M - m0);
#pragma unroll
        for (int c = 0; c < kMaxWidth / 2; ++c)
          if (c < rows) {
            const float f = __fmul_rn(__fmul_rn((float)acc[c], s_xs[half * cols + c]), ws);
            const int64_t o = (int64_t)(m0 + c) * p.ldy + n;
            if (p.out_type == QL_OUT_FP32) {
              reinterpret_cast<float*>(p.y)[o] = p.bias ? f + bias : f;
            } else if (p.out_type == QL_OUT_FP16) {
              __half h = __float2half_rn(f);
              if (p.bias) h = __float2half_rn(__half2float(h) + bias);
              reinterpret_cast<__half*>(p.y)[o] = h;
            } else {
              uint16_t h = f32_to_bf16_rn(f);
              if (p.bias) h = f32_to_bf16_rn(bf16_bits_to_f32(h) + bias);
              reinterpret_cast<uint16_t*>(p.y)[o] = h;
            }
          }
      }
      results_any(false);  // s_xs is read
    }
  } else {
    // ------------------------------------------------------------ weights to f16 in tensor memory
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWiden) : "memory");
    const int q = warp & 3, half = (warp - 12) >> 2;  // lane quadrant; 64 k of a stage's 128
    const int r = 32 * q + lane;
    const uint32_t row = base + (uint32_t)(r * 128);
    const uint32_t to = tmem + ((uint32_t)(32 * q) << 16) + kACol + (uint32_t)(half * 32);
    const uint32_t arrive = in_cta(smem_u32(&ready[0]), 0);
    int s = 0, a = 0, old = 0;  // old: the stage whose A buffer comes next
    uint32_t ph = 0, oph = 0;
    bool ok = true;
    int t, k0, k1;
    int n = 0;  // stages of all items
    for (Walk w(p, pair); w.next(p, t, k0, k1);) n += k1 - k0;
    uint32_t b[16];
    auto load = [&](uint32_t there) {
      if (!__all_sync(0xffffffffu, there) && !wait_warp(&full_w[s], ph, lim, abort)) {
        if (lane == 0) fail();
        ok = false;
        return;
      }
      const uint32_t from = row + (uint32_t)s * kStageBytes;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(b[4 * j]), "=r"(b[4 * j + 1]), "=r"(b[4 * j + 2]), "=r"(b[4 * j + 3])
                     : "r"(from + (uint32_t)(((half * 4 + j) ^ (r & 7)) * 16)));
      if (++s == kStages) {
        s = 0;
        ph ^= 1;
      }
    };
    if (n > 0) load(0);
#pragma unroll 1
    for (int i = 0; i < n && ok; ++i) {
      const uint32_t is_free = ask(&empty[old], oph), there = ask(&full_w[s], ph);
      uint32_t v[32];
#pragma unroll
      for (int j = 0; j < 16; ++j) s8x4_to_f16x2x2(b[j], v[2 * j], v[2 * j + 1]);
      if (i >= kABufs) {
        if (!__all_sync(0xffffffffu, is_free) && !wait_warp(&empty[old], oph, lim, abort)) {
          if (lane == 0) fail();
          break;
        }
        if (++old == kStages) {
          old = 0;
          oph ^= 1;
        }
      }
      tc_fence_after();
      tmem_st_u32x32(to + (uint32_t)a * kACols, v);
      if (i + 1 < n) load(there);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_tmem(arrive + (uint32_t)a * 8);
      if (++a == kABufs) a = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (*abort) {  // set in both CTAs or in neither
    // no copy may land after the pair has left: the last use of every stage is waited for.  Tokens are
    // counted by the first CTA's barriers: for a use of a stage that only one CTA got to, the other
    // half's arrival or bytes are supplied here
    if (threadIdx.x == 0) {
      wait2(&done, 0, kDrainLimit, nullptr);  // no product is reading them
      const int mine = s_issued > s_ahead ? s_issued : s_ahead;
      for (int i = mine > kStages ? mine - kStages : 0; i < mine; ++i)
        wait2(&full_w[i % kStages], (uint32_t)(i / kStages) & 1, kDrainLimit, nullptr);
    }
    if (rank == 0 && threadIdx.x == 0) {
      int other;
      asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(other) : "r"(in_cta(smem_u32(&s_issued), 1)) : "memory");
      const int mine = s_issued, last = mine > other ? mine : other;
      for (int i = last > kStages ? last - kStages : 0; i < last; ++i) {
        uint64_t* bar = &full_x[i % kStages];
        if (i >= mine)
          mbar_arrive_expect_tx(bar, 2 * x_bytes);
        else if (i >= other)
          asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                       "r"(2 * x_bytes)
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

// ------------------------------------------------------------------ tokens to f16
// [M, kpad], zeros past K; 16 codes per thread
__global__ void __launch_bounds__(256) codes_f16_kernel(const int8_t* __restrict__ x, int64_t ldx, int K, int kpad,
                                                        int64_t pieces, uint16_t* __restrict__ img) {
  pdl_wait();
  pdl_launch_dependents();
  const int row = kpad / 16;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / row;
    const int k = (int)(i - m * row) * 16;
    uint32_t h[8] = {};
    if (k < K) {
      const uint4 v = *reinterpret_cast<const uint4*>(x + m * ldx + k);
      s8x4_to_f16x2x2(v.x, h[0], h[1]);
      s8x4_to_f16x2x2(v.y, h[2], h[3]);
      s8x4_to_f16x2x2(v.z, h[4], h[5]);
      s8x4_to_f16x2x2(v.w, h[6], h[7]);
    }
    uint4* to = reinterpret_cast<uint4*>(img + m * kpad + k);
    to[0] = make_uint4(h[0], h[1], h[2], h[3]);
    to[1] = make_uint4(h[4], h[5], h[6], h[7]);
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

bool encode(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t inner, int64_t outer, int64_t row_bytes,
            uint32_t box_inner, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) fprintf(stderr, "qlinear: cuTensorMapEncodeTiled failed (%d)\n", (int)r);
  return r == CUDA_SUCCESS;
}

int64_t kpad_of(int64_t K) { return (K + kStageK - 1) / kStageK * kStageK; }

struct Plan {
  int width, tiles_m, tiles_n, nk, whole, rest, share;
};
Plan plan(int64_t M, int64_t N, int64_t K) {
  Plan c = {};
  const int64_t columns = (M + kMaxWidth - 1) / kMaxWidth;  // of tiles, as few as there can be, evenly wide
  c.width = (int)(((M + columns - 1) / columns + 31) / 32 * 32);
  c.tiles_m = (int)((M + c.width - 1) / c.width);
  c.tiles_n = (int)((N + 255) / 256);
  c.nk = (int)(kpad_of(K) / kStageK);
  const int64_t tiles = (int64_t)c.tiles_m * c.tiles_n;
  c.rest = (int)(tiles % kPairs);
  c.whole = (int)(tiles - c.rest);
  // Equal stretches of the rest, but none so short that joining a tile's parts (3 us, and 0.6 us each)
  // takes longer than it saves of its stages (0.5 us each)
  c.share = (int)(((int64_t)c.rest * c.nk + kPairs - 1) / kPairs);
  int least = 12;
  while (least * least * 5 < 6 * c.nk) ++least;
  if (c.share < least) c.share = least;
  if (c.share > c.nk) c.share = c.nk;
  return c;
}

size_t al256(size_t b) { return (b + 255) & ~size_t(255); }
size_t slot_bytes(const Plan& c) { return al256((size_t)kPairs * 4 * c.width * 128 * 4); }

}  // namespace

size_t codes_gemm_bytes(int64_t M, int64_t N, int64_t K) {
  return slot_bytes(plan(M, N, K)) + al256((size_t)M * kpad_of(K) * 2);
}

cudaError_t launch_codes_gemm(const CodesGemm& g, cudaStream_t st) {
  const Plan c = plan(g.M, g.N, g.K);
  const int64_t kpad = kpad_of(g.K);
  uint16_t* img = reinterpret_cast<uint16_t*>(g.scratch + slot_bytes(c));
  CUtensorMap tw, tx;
  if (!encode(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.w, g.K, g.N, g.ldw, kStageK, 128) ||
      !encode(&tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, img, kpad, g.M, kpad * 2, 64, (uint32_t)c.width / 2))
    return cudaErrorInvalidValue;
  static OncePerDevice once;
  if (const cudaError_t e = raise_smem_limit(codes_gemm_kernel, once); e != cudaSuccess) return e;

  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const int64_t pieces = g.M * kpad / 16, blocks = (pieces + 255) / 256;
  cfg.gridDim = dim3((unsigned)(blocks < 8 * kNumSMs ? blocks : 8 * kNumSMs), 1, 1);
  cudaError_t e = cudaLaunchKernelEx(&cfg, codes_f16_kernel, g.x, g.ldx, (int)g.K, (int)kpad, pieces, img);
  if (e != cudaSuccess) return e;

  Params p = {};
  p.M = (int)g.M;
  p.N = (int)g.N;
  p.nk = c.nk;
  p.width = c.width;
  p.tiles_n = c.tiles_n;
  p.tiles_m = c.tiles_m;
  p.whole = c.whole;
  p.share = c.share;
  p.rest = c.rest;
  p.slots = reinterpret_cast<int32_t*>(g.scratch);
  p.tickets = g.tickets;
  p.x_scale = g.x_scale;
  p.w_scale = g.w_scale;
  p.w_scale_len = g.w_scale_len;
  p.bias = g.bias;
  p.y = g.y;
  p.ldy = g.ldy;
  p.out_type = g.out_type;
  p.status = g.status;
  p.wait_limit = g.wait_limit;
  cfg.gridDim = dim3(2 * kPairs, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = 1024 + (size_t)kStages * kStageBytes;
  return cudaLaunchKernelEx(&cfg, codes_gemm_kernel, tw, tx, p);
}

}  // namespace tc
}  // namespace ql
