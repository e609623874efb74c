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
//   FWD: A = x, B = W13 (both K-major); a tile's columns are half gate, half up columns of the same
//        outputs, so that the activation and the product run in the epilogue and g, u never reach
//        memory (but for the checkpoint)
//   DX : A = [dg du] (K-major), B = W13^T (N-major: H is contiguous)
//   DW : A = [dg du]^T (M-major), B = x^T (N-major)
// A tile is 256 rows by up to 256 columns.
// A pair of CTAs on two SMs shares a tile (cta_group::2): each holds 128 rows of A, half of B's
// columns and 128 rows of the accumulator, so that an SM loads half of B.  The grid is one
// pair per two SMs; pairs take tiles in turn.  Roles in a CTA:
//   warp 0: TMA producer;  warp 1: MMA issue (first CTA of the pair only);  warp 2: tensor memory;
//   warps 4..11: epilogue, one row and half of the columns of the accumulator per thread.
// Two accumulators of 256 columns take turns, so a tile's epilogue runs under the next tile's
// MMAs.
// Where whole tiles would leave most pairs idle in the last round, that round's tiles are cut along
// K into equal parts, one per pair.  A pair that holds a part stores its fp32 sums in a slot of the
// workspace and counts in on the tile's ticket; the CTA that completes the count adds the parts in
// the order of K (the sum does not depend on who is last) and runs the epilogue on them.  Nobody
// waits for another pair.  Equal shares of all tiles of the last two rounds, which would leave no
// pair idle, were slower (4096 x 17408 x 5120 dx: 1009 us against 956 us uncut): the pairs then
// stand at different k and no longer find each other's operands in L2.
// What bounds it: the tensor cores in long calls (4096 tokens, 17408 x 5120: a step 2.38 ms, 1.84
// PFLOP/s, in a burst; 2.6 to 2.7 ms, 1.6 to 1.7, one after the other under the power cap); in
// middling ones (2048 x 2048 x 4096: a step 127 to 130 us, 1.6 PFLOP/s) a step of 64 K takes 0.27 us,
// 0.23 of them the products', and each launch's first loads and last writing about 7 us; in short
// ones those 7 us and the parts' way through L2; the weights' HBM traffic for few tokens (64 x 17408 x
// 5120 forward 65 us, 5.5 TB/s) and the writing of dW13.
// Every wait is bounded; one that runs out raises QL_DEV_TIMEOUT in the status word and the pair
// leaves its loops, waits for copies and MMAs in flight and frees its tensor memory.  Its part of a cut
// tile counts in as missing, so that the next call finds the tickets as it needs them.
#include <cudaTypedefs.h>

#include <cstdio>
#include <mutex>
#include <utility>

#include "common.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace ql {
namespace tc {

namespace {

enum { FWD = 0, DX = 1, DW = 2 };

constexpr int kThreads = 384;
constexpr int kEpiThreads = 256;
constexpr int kBlockK = 64;  // one 128-byte swizzled row of bf16
constexpr int kStages = 6;
constexpr uint32_t kHalfBytes = 128 * kBlockK * 2;  // one operand's half tile of a stage
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr uint32_t kRowStage = 32 * 80;  // an epilogue warp's 32 rows on their way out
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kDrainLimit = 1u << 22;
constexpr int kGroupM = 16;  // tile rows that run before the next tile column

struct Params {
  int rows, cols, K;        // of C; FWD: cols = I (outputs)
  int width;                // columns of a tile: 64, 96, ..., 256
  int tiles_m, tiles_n, nk;
  int whole;                // tiles taken whole, pair after pair
  int cut, parts;           // the tiles after them, each cut along K into so many parts
  float* slots;             // [cut][parts][2 CTAs][64 groups of 4 columns][128 rows][4] sums
  unsigned* tickets;        // [cut tiles][2 CTAs], zero between calls
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
constexpr unsigned kMissing = 1u << 16;  // of a ticket: a part that was not computed
constexpr int64_t kSlotFloats = 256 * 128;  // one CTA's sums of a part

// what a pair works on, one item after the other: whole tiles, then a part of a cut one
struct Walk {
  int t, pair;
  __device__ explicit Walk(int pair) : t(pair), pair(pair) {}
  __device__ bool next(const Params& p, int pairs, int& tile, int& k0, int& k1) {
    if (t < p.whole) {
      tile = t;
      k0 = 0;
      k1 = p.nk;
      t += pairs;
      return true;
    }
    if (pair < 0 || pair >= p.cut * p.parts) return false;
    // neighbouring pairs take the same k of neighbouring tiles
    const int part = pair / p.cut;
    tile = p.whole + pair - part * p.cut;
    k0 = (int)((int64_t)part * p.nk / p.parts);
    k1 = (int)((int64_t)(part + 1) * p.nk / p.parts);
    pair = -1;
    return true;
  }
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
// one lane of a whole warp, the same one every time
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// the whole warp waits; one answer for all lanes
__device__ __forceinline__ bool wait2_warp(uint64_t* bar, uint32_t parity, uint32_t limit, volatile int* abort) {
  return __all_sync(0xffffffffu, wait2(bar, parity, limit, abort));
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

// kind::f16, bf16 operands (format 1), fp32 accumulator, M = 256 over the pair, N = width; bits 15
// and 16: A / B are MN-major
__device__ __forceinline__ uint32_t idesc_pair(bool a_mn, bool b_mn, int width) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(width >> 3) << 17) | ((256u >> 4) << 24);
}

// tile index -> (m, n): blocks of kGroupM tile rows, the rows of a block first
__device__ __forceinline__ void tile_at(const Params& p, int t, int& m, int& n) {
  const int block = t / (kGroupM * p.tiles_n), in = t - block * kGroupM * p.tiles_n;
  const int rows = min(kGroupM, p.tiles_m - block * kGroupM);
  m = block * kGroupM + in % rows;
  n = in / rows;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// One row of BYTES (32 or 64) per lane to global memory through shared memory, so that neighbouring
// lanes write neighbouring 16 bytes: whole sectors instead of 16 bytes of 32 different rows.  dst:
// the first lane's row; rows and bytes of a row that exist.  `stage`: 32 rows of BYTES + 16.
template <int BYTES>
__device__ __forceinline__ void store_rows(uint32_t stage, const uint32_t* w, uint8_t* dst, int64_t pitch, int rows,
                                           int bytes) {
  constexpr int LANES = BYTES / 16, STEP = 32 / LANES;  // lanes per row, rows per store
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < LANES; ++i)
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(stage + lane * (BYTES + 16) + i * 16), "r"(w[4 * i]),
                 "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                 : "memory");
  __syncwarp();
  const int piece = lane % LANES;
#pragma unroll
  for (int i = 0; i < LANES; ++i) {
    const int r = i * STEP + lane / LANES;
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(stage + r * (BYTES + 16) + piece * 16)
                 : "memory");
    if (r < rows && piece * 16 < bytes) *reinterpret_cast<uint4*>(dst + r * pitch + piece * 16) = v;
  }
  __syncwarp();  // read before the next rows are put there
}

__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]),
      "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]),
      "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}

// true in every epilogue thread if `bad` is true in one
__device__ __forceinline__ bool epilogue_any(bool bad) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)bad), "n"(kEpiThreads)
      : "memory");
  return r != 0;
}

// one GEMM on `pairs` pairs of CTAs, of which this is number `pair`
template <int MODE>
__device__ __forceinline__ void gemm(const CUtensorMap& tmA, const CUtensorMap& tmB, const Params& p, int pair,
                                     int pairs) {
  constexpr bool A_MN = MODE == DW, B_MN = MODE != FWD;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], done;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_issued, s_last;
  __shared__ float s_amax[2][2][128][2];  // FWD, int8: [tile parity][column half][row][g, u]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  // the stages start at the same offset in both CTAs
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const int hw = p.width / 2;  // columns of B in each CTA; FWD: outputs of a tile
  const uint32_t lim = p.wait_limit;
  // the epilogue waits for a whole tile's K, the others for a step of it
  const uint32_t lim_tile = (uint32_t)min((uint64_t)lim * (1 + p.nk / 512), (uint64_t)0xFFFFFFFEu);
  volatile int* abort = &s_abort;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 16);  // eight epilogue warps in each CTA
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
  // up to here nothing of the launch before is read or written: this part runs while it ends
  pdl_wait();
  pdl_launch_dependents();
  const uint32_t tmem = s_tmem;
  auto fail = [&]() {
    atomicOr(p.status, (uint32_t)QL_DEV_TIMEOUT);
    *abort = 1;
    st_remote(in_cta(smem_u32(&s_abort), rank ^ 1), 1);
  };

  // The producer and the MMA issuer run as whole warps of which one lane issues: addresses and
  // descriptors then live in uniform registers.  With one lane alone in the loop every operand was
  // moved there anew, and a step of 64 K took 0.35 us whatever was loaded or multiplied in it (the 128
  // steps of 2048 x 2048 x 4096 forward 45.7 us; so 34.6)
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one();
    // bytes of a stage in one CTA: B by N-major chunks of 64 columns is loaded whole
    const uint32_t half_bytes = kHalfBytes + (B_MN ? (hw > 64 ? kHalfBytes : kHalfBytes / 2) : (uint32_t)hw * kBlockK * 2);
    int s = 0, issued = 0;
    uint32_t ph = 1;  // the first pass over the stages finds them empty
    bool ok = true;
    int t, k0, k1;
    for (Walk w(pair); ok && w.next(p, pairs, t, k0, k1);) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int ra = tm * 256 + (int)rank * 128;
      const int rb = MODE == FWD ? tn * hw + (int)rank * p.I : tn * p.width + (int)rank * hw;
      for (int kt = k0; kt < k1; ++kt) {
        if (!wait2_warp(&empty[s], ph, lim, abort)) {
          if (leader) fail();
          ok = false;
          break;
        }
        if (leader) {
          const uint32_t bar = in_cta(smem_u32(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * half_bytes);
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
            if (hw > 64) load_pair(sb + 8192, &tmB, rb + 64, k, bar);
          } else {
            load_pair(sb, &tmB, k, rb, bar);
          }
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
    if (leader) s_issued = issued;
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------------------------------------------------- MMA issue
      const bool leader = elect_one();
      const uint32_t idesc = idesc_pair(A_MN, B_MN, p.width);
      constexpr uint64_t a_step = A_MN ? 2048 / 16 : 2, b_step = B_MN ? 2048 / 16 : 2;  // 16 k
      const uint64_t a0 = A_MN ? desc_mn(base) : smem_desc_sw128(base);
      const uint64_t b0 = B_MN ? desc_mn(base + kHalfBytes) : smem_desc_sw128(base + kHalfBytes);
      int s = 0, n = 0;
      uint32_t ph = 0;
      bool ok = true;
      int t, k0, k1;
      for (Walk w(pair); ok && w.next(p, pairs, t, k0, k1); ++n) {
        const int buf = n & 1;
        if (!wait2_warp(&tempty[buf], (uint32_t)((n >> 1) & 1) ^ 1, lim, abort)) {
          if (leader) fail();
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)buf * 256;
        for (int kt = k0; kt < k1; ++kt) {
          if (!wait2_warp(&full[s], ph, lim, abort)) {
            if (leader) fail();
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = (uint64_t)s * (kStageBytes >> 4);
          if (leader) {
#pragma unroll
            for (int j = 0; j < kBlockK / 16; ++j)
              mma_pair(d, a0 + off + j * a_step, b0 + off + j * b_step, idesc, kt != k0 || j != 0);
            commit_pair(&empty[s]);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (ok && leader) commit_pair(&tfull[buf]);
        __syncwarp();
      }
      if (leader) commit_pair(&done);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 4) >> 2;  // tensor-memory lane quadrant, column half
    const int r = 32 * q + lane;                     // row of this CTA's 128
    const uint32_t stage = base + kStages * kStageBytes + (uint32_t)(warp - 4) * kRowStage;
    // counts a part of cut tile `c` in; true for the last one if every part is there.  That one leaves
    // the ticket at zero for the next call
    auto count_in = [&](int c, unsigned add) {
      unsigned* ticket = p.tickets + 2 * c + rank;
      const unsigned before = atomicAdd(ticket, add);
      if ((before & (kMissing - 1)) != (unsigned)(p.parts - 1)) return false;
      *ticket = 0;
      return before < kMissing;
    };
    bool counted = pair >= p.cut * p.parts;  // no part is this pair's
    int n = 0, t, k0, k1;
    for (Walk w(pair); w.next(p, pairs, t, k0, k1); ++n) {
      int tm, tn;
      tile_at(p, t, tm, tn);
      const int buf = n & 1;
      int got = 0;
      if (lane == 0) got = wait2(&tfull[buf], (uint32_t)(n >> 1) & 1, lim_tile, abort);
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got && lane == 0) fail();
      if (epilogue_any(!got)) break;  // all eight warps or none: they meet at barriers below
      tc_fence_after();
      const int row = tm * 256 + (int)rank * 128 + r;
      const int row0 = row - lane, rows = min(32, p.rows - row0);  // this warp's rows that exist
      const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)buf * 256;

      // a part's sums of this thread's row
      auto slot_of = [&](int part) {
        return p.slots + ((int64_t)((t - p.whole) * p.parts + part) * 2 + rank) * kSlotFloats + r * 4;
      };
      auto load = [&](int c, float (&v)[32]) {  // 32 columns of the tile's sums
        uint32_t u[32];
        tmem_ld_x32(acc + c, u);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
      };
      auto finish = [&]() {
        if constexpr (MODE == FWD) {
          const int i0 = tn * hw, outs = min(hw, p.cols - i0);  // the tile's outputs
          float inv_g = 0.f, inv_u = 0.f;
          const int64_t ipad = ckpt_pad(p.I);
          if (p.save == QL_SAVE_INT8) {
            // first pass over the sums: the largest |g| and |u| of the row's 128 columns (a tile holds
            // one group: its width is 256)
            float ag = 0.f, au = 0.f;
#pragma unroll 1
            for (int c = 64 * half; c < 64 * half + 64; c += 32) {
              float g[32], u[32];
              load(c, g);
              load(hw + c, u);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c + (i & ~7) < outs) {
                  ag = max_nan(ag, fabsf(g[i]));
                  au = max_nan(au, fabsf(u[i]));
                }
            }
            s_amax[buf][half][r][0] = ag;
            s_amax[buf][half][r][1] = au;
            epilogue_any(false);
            ag = max_nan(ag, s_amax[buf][half ^ 1][r][0]);
            au = max_nan(au, s_amax[buf][half ^ 1][r][1]);
            const float sg = ckpt_scale(ag, inv_g), su = ckpt_scale(au, inv_u);
            if (row < p.rows && half == 0) {
              float* s = p.ckpt_scale + (int64_t)row * 2 * (ipad / 128) + tn;
              s[0] = sg;
              s[ipad / 128] = su;
            }
          }
#pragma unroll 1
          for (int c = 64 * half; c < min(64 * half + 64, outs); c += 32) {
            float g[32], u[32];
            load(c, g);
            load(hw + c, u);
            const int left = outs - c;
            if (p.save == QL_SAVE_INT8) {
              uint8_t* ck = reinterpret_cast<uint8_t*>(p.ckpt) + (int64_t)row0 * 2 * ipad + i0 + c;
              uint32_t w[8];
              // (past the last output up to a whole 16 bytes: the padding of the row)
              ckpt_codes32(g, inv_g, w);
              store_rows<32>(stage, w, ck, 2 * ipad, rows, left);
              ckpt_codes32(u, inv_u, w);
              store_rows<32>(stage, w, ck + ipad, 2 * ipad, rows, left);
            }
            uint32_t w[16];
            if (p.save == QL_SAVE_BF16) {
              uint8_t* ck = reinterpret_cast<uint8_t*>(p.ckpt) + ((int64_t)row0 * 2 * ipad + i0 + c) * 2;
#pragma unroll
              for (int j = 0; j < 16; ++j) w[j] = pack2(g[2 * j], g[2 * j + 1]);
              store_rows<64>(stage, w, ck, 4 * ipad, rows, left * 2);
#pragma unroll
              for (int j = 0; j < 16; ++j) w[j] = pack2(u[2 * j], u[2 * j + 1]);
              store_rows<64>(stage, w, ck + 2 * ipad, 4 * ipad, rows, left * 2);
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
              w[j] = pack2(gated_act(g[2 * j], u[2 * j], p.alpha, p.limit),
                           gated_act(g[2 * j + 1], u[2 * j + 1], p.alpha, p.limit));
            store_rows<64>(stage, w, reinterpret_cast<uint8_t*>(p.out + (int64_t)row0 * p.ld_out + i0 + c),
                           p.ld_out * 2, rows, left * 2);
          }
        } else {
          const int c0 = tn * p.width, cols = min(p.width, p.cols - c0);
#pragma unroll 1
          for (int c = 128 * half; c < min(128 * half + 128, cols); c += 32) {
            float v[32];
            load(c, v);
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = pack2(v[2 * j], v[2 * j + 1]);
            store_rows<64>(stage, w, reinterpret_cast<uint8_t*>(p.out + (int64_t)row0 * p.ld_out + c0 + c),
                           p.ld_out * 2, rows, (cols - c) * 2);
          }
        }
      };
      auto release = [&]() {  // the accumulator has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_remote(in_cta(smem_u32(&tempty[buf]), 0));
      };

      if (k1 - k0 == p.nk) {
        finish();
      } else {
        float* dst = slot_of(pair / p.cut);
#pragma unroll 1
        for (int c = 128 * half; c < min(128 * half + 128, p.width); c += 32) {
          float v[32];
          load(c, v);
          if (row < p.rows) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              __stcg(reinterpret_cast<float4*>(dst + (int64_t)(c + i) * 128), make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
          }
          __syncwarp();  // the next read of tensor memory is the whole warp's
        }
        __threadfence();
        epilogue_any(false);  // every warp's part is stored and fenced
        if (threadIdx.x == 128) s_last = count_in(t - p.whole, 1u);
        counted = true;
        epilogue_any(false);
        if (s_last) {
          __threadfence();  // the other parts were fenced before their counts
          // the parts in the order of K, this CTA's own where it stands in it, back to tensor memory
          const int mine = pair / p.cut;
#pragma unroll 1
          for (int c = 128 * half; c < min(128 * half + 128, p.width); c += 32) {
            float v[32], own[32];
            load(c, own);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
#pragma unroll 1
            for (int j = 0; j < p.parts; ++j) {
              if (j == mine) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += own[i];
                continue;
              }
              const float* src = slot_of(j) + (int64_t)c * 128;
              float4 f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                f[i] = row < p.rows ? __ldcg(reinterpret_cast<const float4*>(src + i * 512)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                v[4 * i] += f[i].x;
                v[4 * i + 1] += f[i].y;
                v[4 * i + 2] += f[i].z;
                v[4 * i + 3] += f[i].w;
              }
            }
            tmem_st_x32(acc + c, v);
          }
          tmem_wait_st();
          tc_fence_before();
          epilogue_any(false);  // a row's other half of the columns is another warp's
          tc_fence_after();
          finish();
        }
      }
      release();
    }
    // a pair that gave up counts its part in as missing, and its tile is not finished: the tickets are
    // zero after every launch, whatever ran out
    if (!counted && threadIdx.x == 128) count_in(pair % p.cut, 1u + kMissing);
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
      const uint32_t half_bytes = kHalfBytes + (B_MN ? (hw > 64 ? kHalfBytes : kHalfBytes / 2) : (uint32_t)hw * kBlockK * 2);
      const int mine = s_issued, last = mine > other ? mine : other;
      for (int i = last > kStages ? last - kStages : 0; i < last; ++i) {
        uint64_t* bar = &full[i % kStages];
        if (i >= mine)
          mbar_arrive_expect_tx(bar, half_bytes);
        else if (i >= other)
          asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                       "r"(half_bytes)
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

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ Params p) {
  gemm<MODE>(tmA, tmB, p, blockIdx.x >> 1, gridDim.x >> 1);
}
// dx and dW13 side by side: the first dx_pairs pairs take dx
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ffn_gemms_kernel(const __grid_constant__ CUtensorMap dxA, const __grid_constant__ CUtensorMap dxB,
                     const __grid_constant__ CUtensorMap dwA, const __grid_constant__ CUtensorMap dwB,
                     const __grid_constant__ Params dx, const __grid_constant__ Params dw, int dx_pairs) {
  const int pair = blockIdx.x >> 1;
  if (pair < dx_pairs)
    gemm<DX>(dxA, dxB, dx, pair, dx_pairs);
  else
    gemm<DW>(dwA, dwB, dw, pair - dx_pairs, (gridDim.x >> 1) - dx_pairs);
}

// ------------------------------------------------------------------ gradients of g and u
// dgu[m, i] = dg, dgu[m, I + i] = du from dh and the checkpoint, eight columns of kGradRows rows
// per thread (their loads go out together).  dg and du leave in bf16: the tensor cores multiply bf16
// with bf16, and a second pair of terms for the rest would double both GEMMs.  It moves dx and dW13
// from 0.0017 to 0.0024 of their norm from exact.  One pass over memory: reads dh and the checkpoint,
// writes 4 bytes per output.  Bound by HBM: 4096 x 17408, int8 checkpoint, 570 MB in 104 us, 5.5 TB/s
// (126 us with one row per thread).
constexpr int kGradRows = 4;
template <bool INT8>
__global__ void __launch_bounds__(128) gated_grad_kernel(const uint16_t* __restrict__ dh, int64_t ld_dh, int64_t M,
                                                         int I, const void* __restrict__ ckpt,
                                                         const float* __restrict__ scale, float alpha, float limit,
                                                         uint16_t* __restrict__ dgu) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t ipad = ckpt_pad(I);
  const int i = (blockIdx.x * 128 + threadIdx.x) * 8;
  if (i >= I) return;
  for (int64_t m0 = (int64_t)blockIdx.y * kGradRows; m0 < M; m0 += (int64_t)gridDim.y * kGradRows) {
    uint4 d[kGradRows], kg[kGradRows], ku[kGradRows];
    float sg[kGradRows], su[kGradRows];
#pragma unroll
    for (int r = 0; r < kGradRows; ++r) {
      const int64_t m = min(m0 + r, M - 1);
      d[r] = *reinterpret_cast<const uint4*>(dh + m * ld_dh + i);
      if constexpr (INT8) {
        const int8_t* ck = reinterpret_cast<const int8_t*>(ckpt) + m * 2 * ipad + i;
        const uint2 a = *reinterpret_cast<const uint2*>(ck), b = *reinterpret_cast<const uint2*>(ck + ipad);
        kg[r].x = a.x;
        kg[r].y = a.y;
        ku[r].x = b.x;
        ku[r].y = b.y;
        const float* s = scale + m * 2 * (ipad / 128) + (i >> 7);
        sg[r] = s[0];
        su[r] = s[ipad / 128];
      } else {
        const uint16_t* ck = reinterpret_cast<const uint16_t*>(ckpt) + m * 2 * ipad + i;
        kg[r] = *reinterpret_cast<const uint4*>(ck);
        ku[r] = *reinterpret_cast<const uint4*>(ck + ipad);
      }
    }
#pragma unroll
    for (int r = 0; r < kGradRows; ++r) {
      if (m0 + r >= M) break;
      float g[8], u[8], dv[8], dg[8], du[8];
      if constexpr (INT8) {
        ckpt_values8(make_uint2(kg[r].x, kg[r].y), sg[r], g);
        ckpt_values8(make_uint2(ku[r].x, ku[r].y), su[r], u);
      } else {
        bf16_values8(kg[r], g);
        bf16_values8(ku[r], u);
      }
      bf16_values8(d[r], dv);
#pragma unroll
      for (int j = 0; j < 8; ++j) gated_grad(dv[j], g[j], u[j], alpha, limit, dg[j], du[j]);
      uint16_t* dst = dgu + (m0 + r) * 2 * I + i;
      store8(dst, dg);
      store8(dst + I, du);
    }
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

// Tiles of a GEMM over the pairs: whole ones in turn, and the last round's cut along K where that is
// shorter.  Times in ns, as measured at 2048 x 2048 x 4096: a step of 64 K takes 216 for 64 columns,
// 227 for 128, 247 for 192, 281 for 256 (its waits and issues more than its products); from a tile's
// last product to the end of its writing 1.7 us for 64 and 3.4 for 256, 2.5 and 5.4 with the activation
struct Cut {
  int width, tiles_m, tiles_n, nk, whole, cut, parts;
  int64_t cost;  // of the longest pair
  size_t bytes() const { return (size_t)cut * parts * 2 * kSlotFloats * 4; }
};
constexpr int kPairs = kNumSMs / 2;
int64_t step_ns(int width) { return 190 + width / 3; }
int64_t write_ns(int width, bool fwd) { return fwd ? 1600 + 15 * width : 1100 + 9 * width; }
Cut plan_width(int64_t rows, int64_t cols, int64_t K, int width, bool fwd, int pairs) {
  const int outs = fwd ? width / 2 : width;
  Cut c = {};
  c.width = width;
  c.tiles_m = (int)((rows + 255) / 256);
  c.tiles_n = (int)((cols + outs - 1) / outs);
  c.nk = (int)((K + kBlockK - 1) / kBlockK);
  const int64_t tiles = (int64_t)c.tiles_m * c.tiles_n, step = step_ns(width);
  c.whole = (int)tiles;
  const int rest = (int)(tiles % pairs);
  const int64_t write = write_ns(width, fwd);  // runs under the next tile's products; the last one's does not
  const int64_t whole = c.nk * step > write ? c.nk * step : write;
  int64_t best = (rest ? whole : 0) + write;
  for (int parts = 2; rest > 0 && parts * rest <= pairs && parts <= c.nk && parts <= 8; ++parts) {
    // the longest part, storing it, adding and finishing all parts of a tile by one CTA
    const int64_t ns = (c.nk + parts - 1) / parts * step + write + 3500 + 8 * parts * width;
    if (ns >= best) continue;
    best = ns;
    c.whole = (int)tiles - rest;
    c.cut = rest;
    c.parts = parts;
  }
  c.cost = tiles / pairs * whole + best;
  return c;
}
// Narrower tiles where they fill the rounds better (2048 x 2048 x 4096: 152 tiles of 224 columns in
// two rounds against 128 of 256) or, with few tiles, put more SMs to work; 4 % at least has to come
// of it
Cut plan(int64_t rows, int64_t cols, int64_t K, bool fwd, bool narrow, int pairs = kPairs) {
  Cut c = plan_width(rows, cols, K, 256, fwd, pairs);
  for (int width = 224; narrow && width >= 64; width -= 32) {
    const Cut d = plan_width(rows, cols, K, width, fwd, pairs);
    if (d.cost * 25 < c.cost * 24) c = d;
  }
  return c;
}
// an int8 checkpoint's groups of 128 columns are whole tiles
Cut plan_fwd(int64_t M, int64_t H, int64_t I, bool int8) { return plan(M, I, H, true, !int8); }
Cut plan_dx(int64_t M, int64_t H, int64_t I, int pairs = kPairs) { return plan(M, H, 2 * I, false, true, pairs); }
Cut plan_dw(int64_t M, int64_t H, int64_t I, int pairs = kPairs) { return plan(2 * I, H, M, false, true, pairs); }

// Both gradients in one launch, the pairs shared between them by their work, where neither fills
// the pairs for long: short GEMMs leave them idle at their ends, and a launch is saved.  Past a few
// rounds the two would only take L2 from each other.
struct Both {
  int dx_pairs;  // 0: one GEMM after the other
  Cut dx, dw;
  size_t slots;  // bytes: dx and dW13 alone, one after the other, or together
};
Both make_both(int64_t M, int64_t H, int64_t I) {
  Both b = {0, plan_dx(M, H, I), plan_dw(M, H, I), 0};
  b.slots = b.dx.bytes() > b.dw.bytes() ? b.dx.bytes() : b.dw.bytes();
  auto work = [](const Cut& c) {
    const int64_t k = c.nk * step_ns(c.width), write = write_ns(c.width, false);
    return (int64_t)c.tiles_m * c.tiles_n * (k > write ? k : write);
  };
  const int64_t w0 = work(b.dx), w1 = work(b.dw);
  if (w0 + w1 < 1 || w0 + w1 > (int64_t)12 * kPairs * 64 * 275) return b;  // twelve rounds of 64 steps
  int64_t best = b.dx.cost + b.dw.cost + 3000;  // a launch and a pipeline's start
  const int share = (int)(w0 * kPairs / (w0 + w1));
  for (int d = -6; d <= 14; d += 4) {
    const int n = share + d;
    if (n < 1 || n >= kPairs) continue;
    const Cut x = plan_dx(M, H, I, n), w = plan_dw(M, H, I, kPairs - n);
    const int64_t cost = x.cost > w.cost ? x.cost : w.cost;
    if (cost >= best) continue;
    best = cost;
    b.dx_pairs = n;
    b.dx = x;
    b.dw = w;
  }
  if (b.dx_pairs && b.dx.bytes() + b.dw.bytes() > b.slots) b.slots = b.dx.bytes() + b.dw.bytes();
  return b;
}

// the plan of a thread's last sizes: a call asks for it twice (workspace, launch), a training loop
// again every step, and it takes 1 us on the host
const Both& plan_both(int64_t M, int64_t H, int64_t I) {
  thread_local int64_t at[3] = {-1, -1, -1};
  thread_local Both b;
  if (at[0] != M || at[1] != H || at[2] != I) {
    b = make_both(M, H, I);
    at[0] = M;
    at[1] = H;
    at[2] = I;
  }
  return b;
}

void take(Params& p, const Cut& c) {
  p.width = c.width;
  p.tiles_m = c.tiles_m;
  p.tiles_n = c.tiles_n;
  p.nk = c.nk;
  p.whole = c.whole;
  p.cut = c.cut;
  p.parts = c.parts;
}

template <class... P, class... A>
cudaError_t launch_pdl(void (*kfn)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kfn, std::forward<A>(args)...);
}
constexpr size_t kSmem = 1024 + kStages * kStageBytes + 8 * kRowStage;

template <int MODE>
cudaError_t run(const CUtensorMap& ta, const CUtensorMap& tb, Params& p, const Cut& c, cudaStream_t st) {
  take(p, c);
  static OncePerDevice once;
  if (const cudaError_t e = raise_smem_limit(ffn_gemm_kernel<MODE>, once); e != cudaSuccess) return e;
  const int busy = c.whole > c.cut * c.parts ? c.whole : c.cut * c.parts;
  return launch_pdl(ffn_gemm_kernel<MODE>, dim3(2 * (busy < kPairs ? busy : kPairs)), kThreads, kSmem, st, ta, tb, p);
}

}  // namespace

size_t ffn_forward_slots(int64_t M, int64_t H, int64_t I) {
  const size_t a = plan_fwd(M, H, I, false).bytes(), b = plan_fwd(M, H, I, true).bytes();
  return a > b ? a : b;
}
size_t ffn_backward_slots(int64_t M, int64_t H, int64_t I) {
  return plan_both(M, H, I).slots;
}

void ffn_plan(int gemm, int64_t M, int64_t H, int64_t I, int mode, int32_t* out) {
  Cut c;
  int pairs = kPairs, launches = 1;
  if (gemm == QL_FFN_GEMM_FORWARD) {
    c = plan_fwd(M, H, I, mode == QL_SAVE_INT8);
  } else if (!mode) {
    c = gemm == QL_FFN_GEMM_DX ? plan_dx(M, H, I) : plan_dw(M, H, I);
  } else {
    const Both& b = plan_both(M, H, I);
    c = gemm == QL_FFN_GEMM_DX ? b.dx : b.dw;
    if (!b.dx_pairs)
      launches = 2;
    else
      pairs = gemm == QL_FFN_GEMM_DX ? b.dx_pairs : kPairs - b.dx_pairs;
  }
  out[0] = pairs;
  out[1] = c.width;
  out[2] = c.whole;
  out[3] = c.cut;
  out[4] = c.parts;
  out[5] = launches;
}

cudaError_t launch_ffn_forward(const FfnForward& f, cudaStream_t st) {
  CUtensorMap ta, tb;
  const Cut c = plan_fwd(f.M, f.H, f.I, f.save == QL_SAVE_INT8);
  if (!bf16_map(&ta, f.x, f.H, f.M, f.ldx, 128) ||
      !bf16_map(&tb, f.w13, f.H, 2 * f.I, f.ldw, (uint32_t)(c.width / 2)))
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
  p.slots = f.slots;
  p.tickets = f.tickets;
  return run<FWD>(ta, tb, p, c, st);
}

cudaError_t launch_ffn_backward(const FfnBackward& b, cudaStream_t st) {
  const int64_t gy = (b.M + kGradRows - 1) / kGradRows;
  const dim3 grid((unsigned)((b.I + 1023) / 1024), (unsigned)(gy < 32768 ? gy : 32768));
  const float* scale = b.save == QL_SAVE_INT8 ? b.ckpt_scale : nullptr;
  cudaError_t e = launch_pdl(b.save == QL_SAVE_INT8 ? gated_grad_kernel<true> : gated_grad_kernel<false>, grid, 128, 0,
                             st, b.dh, b.ld_dh, b.M, (int)b.I, b.ckpt, scale, b.alpha, b.limit, b.dgu);
  if (e != cudaSuccess) return e;
  CUtensorMap xa, xb, wa, wb;
  Params x = {}, w = {};
  x.status = w.status = b.status;
  x.wait_limit = w.wait_limit = b.wait_limit;
  x.slots = w.slots = b.slots;
  x.tickets = w.tickets = b.tickets;
  if (b.dx) {
    if (!bf16_map(&xa, b.dgu, 2 * b.I, b.M, 2 * b.I, 128) || !bf16_map(&xb, b.w13, b.H, 2 * b.I, b.ldw, 64))
      return cudaErrorInvalidValue;
    x.rows = (int)b.M;
    x.cols = (int)b.H;
    x.K = (int)(2 * b.I);
    x.out = b.dx;
    x.ld_out = b.ld_dx;
  }
  if (b.dw13) {
    if (!bf16_map(&wa, b.dgu, 2 * b.I, b.M, 2 * b.I, 64) || !bf16_map(&wb, b.x, b.H, b.M, b.ldx, 64))
      return cudaErrorInvalidValue;
    w.rows = (int)(2 * b.I);
    w.cols = (int)b.H;
    w.K = (int)b.M;
    w.out = b.dw13;
    w.ld_out = b.ld_dw;
  }
  if (!b.dw13) return run<DX>(xa, xb, x, plan_dx(b.M, b.H, b.I), st);
  if (!b.dx) return run<DW>(wa, wb, w, plan_dw(b.M, b.H, b.I), st);
  const Both& both = plan_both(b.M, b.H, b.I);
  if (!both.dx_pairs) {
    e = run<DX>(xa, xb, x, both.dx, st);
    return e != cudaSuccess ? e : run<DW>(wa, wb, w, both.dw, st);
  }
  take(x, both.dx);
  take(w, both.dw);
  w.slots += both.dx.bytes() / sizeof(float);
  w.tickets += 2 * kPairs;
  static OncePerDevice once;
  e = raise_smem_limit(ffn_gemms_kernel, once);
  if (e != cudaSuccess) return e;
  return launch_pdl(ffn_gemms_kernel, dim3(2 * kPairs), kThreads, kSmem, st, xa, xb, wa, wb, x, w, both.dx_pairs);
}

}  // namespace tc
}  // namespace ql
