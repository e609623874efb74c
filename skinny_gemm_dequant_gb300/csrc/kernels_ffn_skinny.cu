// The gated feed-forward block on bf16 weights for few tokens, streaming the weights once:
//   h = silu(a min(g, L)) clamp(u, -L, L),  g = x Wg^T, u = x Wu^T
//
// bf16 products are exact in fp32 and the warp MMA sums them in fp32; g and u stay there until the
// activation.  The weights are the MMA's A operand (16 rows), the tokens its N = 8 columns.  A CTA
// owns 16 outputs: 16 gate rows and the matching 16 up rows; its warps take K in turn, 32 at a time
// (64 bytes of every row), and their sums meet in shared memory.  Which k an MMA slot stands for is
// free as long as both operands agree: a lane's 16-byte piece of a row is four slots.  Every lane
// copies its own pieces, of weights and activations, to its own slots of a ring (cp.async), so a
// warp needs no barrier.  (Activations read where they are used, or a block ahead into registers:
// 13 x 17408 x 5120 62.9 us, so 60.8; 1 x 2056 x 4096 8.5 and 7.3.)
//
// Bound by HBM for large weights: 1 token x 17408 x 5120 (356 MB) 54.2 us, 6.6 TB/s, 0.97 of the
// measured copy rate; 13 x 2056 x 4096 (34 MB) 8.3 us, where launch, first loads and the joining of
// the K shares are half of it.

#include "common.cuh"
#include "ffn.h"
#include "ffn_act.cuh"
#include "internal.h"

namespace ql {

namespace {

constexpr int kBlockK = 32;      // k per block
constexpr int kPrefetch = 2;  // blocks
constexpr int kOut = 16;         // outputs of a CTA
constexpr uint32_t kWBlock = 4 * 512;  // a warp's weight bytes per block: 32 rows of 64

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

// NT: 8-token tiles; kDepth: blocks in a warp's ring.  gridDim.z CTAs (a cluster) split K further.
template <int NT, int kDepth, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) ffn_skinny_kernel(const __grid_constant__ FfnSkinnyArgs a) {
  constexpr int TT = NT * 8, PITCH = TT + 1, kThreads = kWarps * 32;
  constexpr uint32_t kBlock = kWBlock + NT * 512;  // and the activations'
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
  // the end are zeros: neither is stored
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
    xp[nt] = a.x + (int64_t)(m0 + nt * 8 + g) * a.ldx + (int64_t)b0 * kBlockK + t * 8;

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
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        cp16(mine + slot * kBlock + kWBlock + nt * 512, xp[nt], take && nt * 8 + g < toks);
        xp[nt] += bstep * kBlockK;
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

  uint32_t slot = 0;
  for (int b = b0; b < nblk; b += bstep) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
    uint4 wv[2][2];
#pragma unroll
    for (int up = 0; up < 2; ++up)
#pragma unroll
      for (int h = 0; h < 2; ++h) wv[up][h] = lds16(mine + slot * kBlock + (up * 2 + h) * 512);
    uint4 xv[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xv[nt] = lds16(mine + slot * kBlock + kWBlock + nt * 512);
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

template <int NT, int kDepth, int kWarps>
cudaError_t launch(const FfnSkinnyArgs& a, cudaStream_t st) {
  auto* kfn = ffn_skinny_kernel<NT, kDepth, kWarps>;
  static OncePerDevice once;
  if (const cudaError_t e = raise_smem_limit(kfn, once); e != cudaSuccess) return e;
  const dim3 grid((unsigned)((a.N + kOut - 1) / kOut), (unsigned)((a.M + NT * 8 - 1) / (NT * 8)));
  // K over a cluster's CTAs while all of them find a place at once (16 warps per SM; 96 x 1024 x 2048 in
  // two waves 14.9 us, unsplit 8.6) and every warp keeps four blocks or more (13 x 2056 x 4096, 8 warps:
  // 2 CTAs 9.1 us, 1: 9.7, 4: 13.0)
  const int nblk = (a.K + kBlockK - 1) / kBlockK;
  int ks = 1;
  while (ks < 8 && (int64_t)grid.x * grid.y * ks * kWarps <= 8 * kNumSMs && nblk >= kWarps * ks * 8) ks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid.x, grid.y, (unsigned)ks);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = kWarps * kDepth * (kWBlock + NT * 512);
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
  // up to a CTA per SM, 16 warps share its K: 13 x 2056 x 4096 8.3 us, with 8 warps and a cluster of two
  // 9.1 (32 tokens 10.1 and 11.6); at 13 x 4096 x 2048 (256 CTAs) 10.1 and 8.2.  They want four
  // blocks each (1 x 520 x 1024: 2.5 us, 8 warps 2.3).  32 tokens: three blocks in the ring let two
  // CTAs on an SM (73 us against 82 with four at 17408 x 5120)
  const bool few = (int64_t)((a.N + kOut - 1) / kOut) * ((a.M + 31) / 32) <= kNumSMs && a.K > 63 * kBlockK;
  if (a.M <= 8) return few ? launch<1, 3, 16>(a, st) : launch<1, 4, 8>(a, st);
  if (a.M <= 16) return few ? launch<2, 3, 16>(a, st) : launch<2, 4, 8>(a, st);
  return few ? launch<4, 3, 16>(a, st) : launch<4, 3, 8>(a, st);
}

}  // namespace ql
