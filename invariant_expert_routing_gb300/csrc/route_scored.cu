// Routing by scores (sigmoid or softmax) with a selection bias, expert groups
// and renormalised, scaled gates.
//
// Per token, one warp, expert e = lane + 32 s in register s of a lane:
//   score_e = 1 / (1 + exp(-l_e))  or  exp(l_e - m) / sum_i exp(l_i - m)
//   b_e = score_e + bias_e                       (selection only)
//   groups of N / G consecutive experts rank by the largest b or by the sum
//   of the two largest; the best `top_groups` stay
//   the k largest b of the experts that stay; slots in ascending expert order
//   gate_j = scale * score_j [/ (sum of the selected scores + 1e-20)]
// Ties go to the lower index, NaN ranks last.  Values are ranked through
// order-preserving 32-bit keys, so that the warp-wide maximum is one redux
// instruction and a round of the top-k two (largest key, then the lowest
// expert among the lanes that hold it).
#include <cmath>
#include <cstdint>

#include "kernels.h"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kSlots = 8;         // experts a lane: N <= 256
constexpr int kMaxGroups = 32;
constexpr int kRouteWarps = 8;

// Larger floats have larger keys; +0 and -0 are equal; NaN is 1, below every
// number; 0 is left for "not available".
__device__ __forceinline__ uint32_t key_of(float f) {
  if (isnan(f)) return 1u;
  const uint32_t b = __float_as_uint(f + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  if (key <= 1u) return NAN;
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

__global__ void __launch_bounds__(32 * kRouteWarps) route_scored_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias, int T, int N, int k, int sigmoid, int groups,
    int top_groups, int top2, int renormalize, float scale, int32_t* __restrict__ idx_out,
    float* __restrict__ gate_out) {
  __shared__ uint32_t s_key[kRouteWarps][32 * kSlots];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long t = (long long)blockIdx.x * kRouteWarps + warp;
  pdl_wait();
  pdl_trigger();
  if (t >= T) return;
  constexpr uint32_t kAll = 0xffffffffu;
  const float* row = logits + t * N;
  float sc[kSlots];
  uint32_t key[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) sc[s] = lane + 32 * s < N ? __ldg(row + lane + 32 * s) : -INFINITY;
  if (sigmoid) {
#pragma unroll
    for (int s = 0; s < kSlots; ++s) sc[s] = 1.0f / (1.0f + expf(-sc[s]));
  } else {
    float m = sc[0];
#pragma unroll
    for (int s = 1; s < kSlots; ++s) m = fmaxf(m, sc[s]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
    if (m == -INFINITY) m = 0.0f;   // every logit is -inf (or NaN): scores 0 (NaN)
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      sc[s] = expf(sc[s] - m);
      sum += sc[s];
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
    if (sum == 0.0f) sum = 1.0f;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) sc[s] = sc[s] / sum;
  }
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int e = lane + 32 * s;
    key[s] = e < N ? key_of(bias ? sc[s] + __ldg(bias + e) : sc[s]) : 0u;
  }

  if (groups > 1) {
    // lane g: the two best of group g, then its rank among the groups
    const int size = N / groups;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) s_key[warp][lane + 32 * s] = key[s];
    __syncwarp();
    uint32_t gkey = 0;
    if (lane < groups) {
      uint32_t a = 0, b = 0;
      for (int i = 0; i < size; ++i) {
        const uint32_t q = s_key[warp][lane * size + i];
        b = max(b, min(a, q));
        a = max(a, q);
      }
      gkey = top2 ? key_of(value_of(a) + value_of(b)) : a;
    }
    int better = 0;
    for (int g = 0; g < groups; ++g) {
      const uint32_t o = __shfl_sync(kAll, gkey, g);
      better += (o > gkey || (o == gkey && g < lane)) ? 1 : 0;
    }
    const unsigned kept = __ballot_sync(kAll, lane < groups && better < top_groups);
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const int e = lane + 32 * s;
      if (e < N && !((kept >> (e / size)) & 1u)) key[s] = 0u;
    }
  }

  uint32_t chosen = 0;   // bit s: expert lane + 32 s is selected
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int s = kSlots - 1; s >= 0; --s) {
      if (key[s] >= best) {
        best = key[s];
        at = s;
      }
    }
    const uint32_t top = __reduce_max_sync(kAll, best);
    const uint32_t e = best == top ? (uint32_t)(lane + 32 * at) : 0xffffu;
    const uint32_t win = __reduce_min_sync(kAll, e);
    if (e == win) {
      chosen |= 1u << at;
#pragma unroll
      for (int s = 0; s < kSlots; ++s)
        if (s == at) key[s] = 0u;
    }
  }

  float sum = 0.0f;
  unsigned mask[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    mask[s] = __ballot_sync(kAll, (chosen >> s) & 1u);
    if (renormalize)
      for (unsigned m = mask[s]; m != 0u; m &= m - 1u) sum += __shfl_sync(kAll, sc[s], __ffs(m) - 1);
  }
  const float div = renormalize ? sum + 1e-20f : 1.0f;
  int base = 0;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if ((chosen >> s) & 1u) {
      const int slot = base + __popc(mask[s] & ((1u << lane) - 1u));
      idx_out[t * k + slot] = lane + 32 * s;
      gate_out[t * k + slot] = scale * (sc[s] / div);
    }
    base += __popc(mask[s]);
  }
}

}  // namespace

int route_scored_max_groups() { return kMaxGroups; }

void launch_route_scored(const float* logits, const float* bias, int T, int N, int k, bool sigmoid, int groups,
                         int top_groups, bool top2, bool renormalize, float scale, int32_t* topk_idx,
                         float* topk_gate, cudaStream_t s) {
  launch_pdl(route_scored_kernel, dim3((T + kRouteWarps - 1) / kRouteWarps), dim3(32 * kRouteWarps), 0, s, logits,
             bias, T, N, k, sigmoid ? 1 : 0, groups, top_groups, top2 ? 1 : 0, renormalize ? 1 : 0, scale, topk_idx,
             topk_gate);
}

}  // namespace moe
