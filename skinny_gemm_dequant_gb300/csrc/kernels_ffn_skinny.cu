// The gated feed-forward block on bf16 weights for few tokens, streaming the weights once:
//   h = silu(a min(g, L)) clamp(u, -L, L),  g = x Wg^T, u = x Wu^T
//
// bf16 products are exact in fp32 and the warp MMA sums them in fp32; g and u stay there until the
// activation.  The weights are the MMA's A operand (16 rows), the tokens its N = 8 columns.  A CTA
// owns 16 outputs: 16 gate rows and the matching 16 up rows; its eight warps take K in turn, 32 at
// a time (64 bytes of every row), and their sums meet in shared memory.  Which k an MMA slot stands
// for is free as long as both operands agree: a lane's 16-byte piece of a row is four slots.  Every
// lane copies its own pieces (cp.async) to its own slots of a ring, so a warp needs no barrier.
//
// Bound by HBM for large weights: 1 token x 17408 x 5120 (356 MB) 55.6 us, 6.4 TB/s, 0.94 of the
// measured copy rate; 13 x 2056 x 4096 (34 MB) 9.3 us, where launch, first loads and the joining of
// the K shares are half of it.
#include <atomic>

#include "common.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "internal.h"

namespace ql {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kDepth = 4;        // blocks in a warp's ring
constexpr int kBlockK = 32;      // k per block
constexpr int kPrefetch = 2;  // blocks
constexpr int kOut = 16;         // outputs of a CTA
constexpr uint32_t kBlock = 4 * 512;  // a warp's bytes per block: 32 rows of 64

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

// NT: 8-token tiles.  gridDim.z CTAs (a cluster) split K further.
template <int NT>
__global__ void __launch_bounds__(kThreads) ffn_skinny_kernel(const __grid_constant__ FfnSkinnyArgs a) {
  constexpr int TT = NT * 8, PITCH = TT + 1;
  extern __shared__ __align__(16) uint8_t ring[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int m0 = blockIdx.y * TT, toks = min(TT, a.M - m0);
  const int n0 = blockIdx.x * kOut;
  const int ks = gridDim.z, kz = blockIdx.z;
  const int nblk = (a.K + kBlockK - 1) / kBlockK;
  const int b0 = kz * kWarps + warp, bstep = ks * kWarps;
  const uint32_t mine = smem_addr(ring) + (uint32_t)warp * (kDepth * kBlock) + (uint32_t)lane * 16;

  // this lane's rows, [gate, up][half of the 16]; rows past the end read the last row, tokens past
  // the end the last token: neither is stored
  const uint8_t* wp[2][2];
#pragma unroll
  for (int up = 0; up < 2; ++up)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t n = min(n0 + h * 8 + g, a.N - 1);
      wp[up][h] = a.w + (up ? a.N + n : n) * a.ldw_bytes + (int64_t)b0 * 64 + t * 16;
    }
  const uint16_t* xp[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    xp[nt] = a.x + (int64_t)(m0 + min(nt * 8 + g, toks - 1)) * a.ldx + (int64_t)b0 * kBlockK + t * 8;

  int bf = b0;  // the next block to fetch
  auto fetch = [&](uint32_t slot) {
    if (bf < nblk) {
      const bool take = bf * kBlockK + t * 8 < a.K;
#pragma unroll
      for (int up = 0; up < 2; ++up)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          cp16(mine + slot * kBlock + (up * 2 + h) * 512, wp[up][h], take);
          wp[up][h] += bstep * 64;
        }
      bf += bstep;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // Before the wait for the launch before, nothing is read or written but L2 is asked for the first
  // blocks' rows (a prefetch only moves them there): a row per lane
  if (n0 + lane % kOut < a.N) {
    const uint8_t* row = a.w + ((lane >= kOut ? (int64_t)a.N : 0) + n0 + lane % kOut) * a.ldw_bytes;
    for (int d = 0, b = b0; d < kPrefetch && b < nblk; ++d, b += bstep) prefetch_l2(row + (int64_t)b * 64);
  }
  pdl_wait();
#pragma unroll
  for (int d = 0; d < kDepth - 1; ++d) fetch(d);

  float acc[2][NT][4];
#pragma unroll
  for (int up = 0; up < 2; ++up)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[up][nt][i] = 0.f;

  // activations; more than 8 tokens' a block ahead (13 x 2056 x 4096: 10.4 to 9.4 us, 16 x 17408 x
  // 5120: 68.1 to 63.3 us; 8 tokens 58.3 to 60.0 us)
  uint4 x_next[NT];
  auto x_load = [&](int b) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      x_next[nt] = make_uint4(0u, 0u, 0u, 0u);
      if (b < nblk && b * kBlockK + t * 8 < a.K) x_next[nt] = *reinterpret_cast<const uint4*>(xp[nt]);
      xp[nt] += bstep * kBlockK;
    }
  };
  if constexpr (NT > 1) x_load(b0);
  uint32_t slot = 0;
  for (int b = b0; b < nblk; b += bstep) {
    if constexpr (NT == 1) x_load(b);  // before the wait for the weights: the latencies overlap
    uint4 xv[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xv[nt] = x_next[nt];
    if constexpr (NT > 1) x_load(b + bstep);
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
    uint4 wv[2][2];
#pragma unroll
    for (int up = 0; up < 2; ++up)
#pragma unroll
      for (int h = 0; h < 2; ++h) wv[up][h] = lds16(mine + slot * kBlock + (up * 2 + h) * 512);
    // the slot of the block before this one is free: its pieces are in registers
    fetch(slot == 0 ? kDepth - 1 : slot - 1);
    if (++slot == kDepth) slot = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int up = 0; up < 2; ++up) {
        mma_bf16_16816(acc[up][nt], wv[up][0].x, wv[up][1].x, wv[up][0].y, wv[up][1].y, xv[nt].x, xv[nt].y);
        mma_bf16_16816(acc[up][nt], wv[up][0].z, wv[up][1].z, wv[up][0].w, wv[up][1].w, xv[nt].z, xv[nt].w);
      }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  pdl_launch_dependents();  // the next launch may take the places that become free

  // every warp leaves its sums in its own part of the ring (its copies have landed and are read).
  // Accumulator i of lane (g, t): row g + 8 (i >> 1), token 2t + (i & 1)
  static_assert(2 * kOut * PITCH * 4 <= kDepth * kBlock, "a warp's sums fit its part of the ring");
  auto sums = [&](int w) { return reinterpret_cast<float*>(ring + w * (kDepth * kBlock)); };
  __syncwarp();
#pragma unroll
  for (int up = 0; up < 2; ++up)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sums(warp)[(up * kOut + g + 8 * (i >> 1)) * PITCH + nt * 8 + 2 * t + (i & 1)] = acc[up][nt][i];
  __syncthreads();
  auto cta_total = [&](int r, int m) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += sums(w)[r * PITCH + m];
    return v;
  };
  if (ks > 1) {
    // the CTA's own sums first, into warp 0's part: each value is read and replaced by one thread
    for (int e = threadIdx.x; e < 2 * kOut * toks; e += kThreads) {
      const int r = e % (2 * kOut), m = e / (2 * kOut);
      sums(0)[r * PITCH + m] = cta_total(r, m);
    }
    __syncthreads();
    cluster_sync_all();
  }
  auto total = [&](int r, int m) {
    if (ks == 1) return cta_total(r, m);
    float v = 0.f;
    for (int z = 0; z < ks; ++z) v += ld_cta(smem_addr(sums(0) + r * PITCH + m), (uint32_t)z);
    return v;
  };
  // the CTAs of a cluster share the outputs
  for (int e = kz * kThreads + threadIdx.x; e < kOut * toks; e += ks * kThreads) {
    const int o = e % kOut, m = e / kOut;
    if (n0 + o < a.N)
      a.y[(int64_t)(m0 + m) * a.ldy + n0 + o] =
          f32_to_bf16_rn(gated_act(total(o, m), total(kOut + o, m), a.alpha, a.limit));
  }
  if (ks > 1) cluster_sync_all();  // the others may still read this CTA's sums
}

template <int NT>
cudaError_t launch(const FfnSkinnyArgs& a, cudaStream_t st) {
  auto* kfn = ffn_skinny_kernel<NT>;
  static std::atomic<int> attr{0};
  if (!attr.load()) {
    cudaError_t e = raise_smem_limit(kfn);
    // the activations live in L1, so not all of it goes to the rings: 8 x 17408 x 5120 57.1 us with
    // half, 60.6 with none of it left; 16 tokens 66.9 us with a fifth, 69.7 with half (registers keep
    // the CTAs few); 32 tokens 74.0 and 95.3 us; 1 token 55.3 and 54.5 us
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kfn, cudaFuncAttributePreferredSharedMemoryCarveout, NT == 2 ? 80 : 50);
    if (e != cudaSuccess) return e;
    attr.store(1);
  }
  const dim3 grid((unsigned)((a.N + kOut - 1) / kOut), (unsigned)((a.M + NT * 8 - 1) / (NT * 8)));
  // K over a cluster's CTAs while there are fewer than three CTAs per two SMs and every warp keeps
  // four blocks or more (13 x 2056 x 4096: 2 CTAs 10.9 us, 1: 15.8, 4: 14.9)
  const int nblk = (a.K + kBlockK - 1) / kBlockK;
  int ks = 1;
  while (ks < 8 && (int64_t)grid.x * grid.y * ks < 3 * kNumSMs / 2 && nblk >= kWarps * ks * 8) ks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid.x, grid.y, (unsigned)ks);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kWarps * kDepth * kBlock;
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
  return cudaLaunchKernelEx(&cfg, kfn, a);
}

}  // namespace

cudaError_t launch_ffn_skinny(const FfnSkinnyArgs& a, cudaStream_t st) {
  if (a.M <= 8) return launch<1>(a, st);
  if (a.M <= 16) return launch<2>(a, st);
  return launch<4>(a, st);
}

}  // namespace ql
