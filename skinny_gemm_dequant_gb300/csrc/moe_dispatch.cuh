// Routing and dispatch of the mixture-of-experts launches, and what GATE_UP hands to DOWN.
#pragma once
#include "common.cuh"
#include "route.cuh"
#include "stream.h"
#include "stream_dev.cuh"

namespace ql {

constexpr int kPerEntry = 8;  // pairs: one token tile of the products

// Routing and dispatch, by every CTA for itself: pairs sorted by (expert, how often the token had it
// before), entries of up to `most` pairs.  Scratch: P keys.
struct Lists {
  Entry* entries;
  int* ids;        // by pair
  uint16_t *pair, *tok;  // sorted
  Entry* heads;    // scratch
  int* keys;       // scratch
};

// what GATE_UP hands to DOWN beside h
struct Handed {
  static constexpr int kPairs = kMoeMaxTokens * kMoeMaxTopk;
  int entries, most, pad[2];
  Entry entry[kPairs];
  float weight[kPairs];  // by pair
  uint16_t pair[kPairs], tok[kPairs];
};
static_assert(sizeof(Handed) <= kMoeHandedBytes, "workspace");

// by one warp of one CTA: the lists
__device__ __forceinline__ void hand_lists(const StreamArgs& p, const Lists& l, int entries, int most) {
  Handed& to = *reinterpret_cast<Handed*>(p.handed);
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    to.entries = entries;
    to.most = most;
  }
  for (int i = lane; i < p.M * p.topk; i += 32) {
    if (i < entries) to.entry[i] = l.entries[i];
    to.pair[i] = l.pair[i];
    to.tok[i] = l.tok[i];
  }
}
// by one warp: the weights of token m (and the call's outputs of its routing)
__device__ __forceinline__ void hand_weights(const StreamArgs& p, const Lists& l, int m) {
  const int lane = threadIdx.x & 31;
  int id = 0;
  float wt = 0.f;
  if (p.logits)
    route_token_warp(p.logits + (int64_t)m * p.E, p.E, p.topk, p.renorm != 0, id, wt);
  else if (lane < p.topk)
    wt = p.wts[m * p.topk + lane];
  if (lane < p.topk) {
    const int i = m * p.topk + lane;
    reinterpret_cast<Handed*>(p.handed)->weight[i] = wt;
    if (p.wts_out) p.wts_out[i] = wt;
    if (p.ids_out) p.ids_out[i] = l.ids[i] == kNone ? -1 : l.ids[i];
  }
}

__device__ __forceinline__ void route(const StreamArgs& p, const Lists& l, int warps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
  for (int m = warp; m < p.M; m += warps) {
    int id = -1;
    float wt;
    if (p.logits)
      route_token_warp<false>(p.logits + (int64_t)m * p.E, p.E, p.topk, false, id, wt);
    else if (lane < p.topk)
      id = p.ids[m * p.topk + lane];
    if (id < 0 || id >= p.E) id = kNone;  // padding: not dispatched
    if (lane < p.topk) l.ids[m * p.topk + lane] = id;
  }
}

// One token, by one warp: an entry for each pair.  Returns their number.
__device__ __forceinline__ int route_one(const StreamArgs& p, const Lists& l) {
  const int lane = threadIdx.x & 31;
  int id = -1;
  float wt;
  if (p.logits)
    route_token_warp<false>(p.logits, p.E, p.topk, false, id, wt);
  else if (lane < p.topk)
    id = p.ids[lane];
  const bool on = lane < p.topk && id >= 0 && id < p.E;
  const unsigned all = __ballot_sync(0xffffffffu, on);
  if (lane < p.topk) l.ids[lane] = on ? id : kNone;
  if (on) {
    const int n = __popc(all & ((1u << lane) - 1));
    l.entries[n] = {(uint16_t)id, (uint16_t)n, 1};
    l.pair[n] = (uint16_t)lane;
    l.tok[n] = 0;
  }
  return __popc(all);
}

// after a barrier; ends with one.  Returns the number of entries, and the most pairs of one
template <int WARPS>
__device__ __forceinline__ int dispatch(const StreamArgs& p, const Lists& l, int per_entry, int& most_out) {
  __shared__ int s_entries, s_most;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, P = p.M * p.topk;
#pragma unroll 1
  for (int i = threadIdx.x; i < P; i += WARPS * 32) {
    int repeats = 0;
    if (!p.logits)
      for (int j = i - i % p.topk; j < i; ++j) repeats += l.ids[j] == l.ids[i];
    l.keys[i] = l.ids[i] == kNone ? kNone : l.ids[i] * kMoeMaxTopk + repeats;
  }
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < P; i += WARPS * 32) {
    const int key = l.keys[i];
    int before = 0, rank = 0, all = 0;
    auto meet = [&](int o, int j) {
      before += o < key;
      all += o == key;
      rank += o == key && j < i;
    };
    int j = 0;
#pragma unroll 2
    for (; j + 4 <= P; j += 4) {
      const int4 o = *reinterpret_cast<const int4*>(l.keys + j);
      meet(o.x, j);
      meet(o.y, j + 1);
      meet(o.z, j + 2);
      meet(o.w, j + 3);
    }
    for (; j < P; ++j) meet(l.keys[j], j);
    l.pair[before + rank] = (uint16_t)i;
    l.tok[before + rank] = (uint16_t)(i / p.topk);
    const bool head = key != kNone && rank % per_entry == 0;
    l.heads[before + rank] = {(uint16_t)l.ids[i], (uint16_t)(before + rank), head ? min(per_entry, all - rank) : 0};
  }
  __syncthreads();
  if (warp == 0) {
    int n = 0, most = 1;
#pragma unroll 1
    for (int i0 = 0; i0 < P; i0 += 32) {
      const int count = i0 + lane < P ? l.heads[i0 + lane].count : 0;
      const unsigned all = __ballot_sync(0xffffffffu, count > 0);
      most = max(most, count);
      if (count > 0) l.entries[n + __popc(all & ((1u << lane) - 1))] = l.heads[i0 + lane];
      n += __popc(all);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      s_entries = n;
      s_most = most;
    }
  }
  __syncthreads();
  most_out = s_most;
  return s_entries;
}

}  // namespace ql
