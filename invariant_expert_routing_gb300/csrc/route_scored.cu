// Routing by scores (sigmoid or softmax) with a selection bias, expert groups
// and renormalised, scaled gates.
//
// Per token:
//   score_e = 1 / (1 + exp(-l_e))  or  exp(l_e - m) / sum_i exp(l_i - m)
//   b_e = score_e + bias_e                       (selection only)
//   groups of N / G consecutive experts rank by the largest b or by the sum
//   of the two largest; the best `top_groups` stay
//   the k largest b of the experts that stay; slots in ascending expert order
//   gate_j = scale * score_j [/ (sum of the selected scores + 1e-20)]
// Ties go to the lower index, NaN ranks last.
//
// Two kernels, by N and the groups alone.  Where a lane can hold 4, 8 or 16
// consecutive experts of one group, half a warp takes a token: each lane sorts
// its four best values (no indices), group scores are a merge of the lanes'
// first two, and a round of the top-k is a maximum over the lanes, a ballot and
// a shift of the winner's list, without a scan of the lane's experts; two tokens
// share every instruction (131072 tokens, 256 experts, 8 groups: 70.4 us; a
// whole warp per token took 20 more).  Any other shape, and a token with a NaN
// or +inf value or fewer than k values above -inf, takes experts lane + 32 s
// and scans, ranking through order-preserving integer keys (every token so, after
// the lanes gave it up: 304 us).  Bound by instruction issue; the scores alone
// (an exponential and a reciprocal per expert) are a fifth.
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

// Four times the sigmoid: the reciprocal is taken of a quarter of 1 + exp(-l), so that it is a
// normal number wherever the exponential is finite, and the factor of a quarter, applied where
// scores are used, brings the subnormal scores between l = -88.7 and -87.3, which still rank.
// (131072 tokens x 256 experts: 69.9 us, 69.0 without, 70.8 with the factor here, 73.6 with a reciprocal that
// handles subnormals itself.)  The exponential is accurate, the reciprocal off by one unit at
// most, 0 for an infinite argument (l below -88.7).
__device__ __forceinline__ float sigmoid4(float l) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(0.25f, expf(-l), 0.25f)));
  return r;
}
__device__ __forceinline__ float score_unit(int sigmoids) { return sigmoids ? 0.25f : 1.0f; }

// Scores of a lane's E experts from its logits (absent experts: -inf), W lanes a token, in units
// of score_unit.
template <int W, int E>
__device__ __forceinline__ void scores_of(float (&sc)[E], int sigmoids) {
  constexpr uint32_t kAll = 0xffffffffu;
  if (sigmoids) {
#pragma unroll
    for (int s = 0; s < E; ++s) sc[s] = sigmoid4(sc[s]);
    return;
  }
  float m = sc[0];
#pragma unroll
  for (int s = 1; s < E; ++s) m = fmaxf(m, sc[s]);
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
  if (m == -INFINITY) m = 0.0f;   // every logit is -inf (or NaN): scores 0 (NaN)
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < E; ++s) {
    sc[s] = expf(sc[s] - m);
    sum += sc[s];
  }
#pragma unroll
  for (int off = W / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
  const float inv = sum == 0.0f ? 1.0f : 1.0f / sum;
#pragma unroll
  for (int s = 0; s < E; ++s) sc[s] *= inv;
}

// One token by a warp, experts lane + 32 s, any groups and any values.
// s_key: 256 words of the warp.
__device__ __noinline__ void route_row(const float* __restrict__ row, const float* __restrict__ bias, int N, int k,
                                       int sigmoids, int groups, int top_groups, int top2, int renormalize,
                                       float scale, uint32_t* s_key, int32_t* __restrict__ idx_out,
                                       float* __restrict__ gate_out) {
  const int lane = threadIdx.x & 31;
  constexpr uint32_t kAll = 0xffffffffu;
  float sc[kSlots];
  uint32_t key[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) sc[s] = lane + 32 * s < N ? __ldg(row + lane + 32 * s) : -INFINITY;
  scores_of<32, kSlots>(sc, sigmoids);
  const float unit = score_unit(sigmoids);
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    const int e = lane + 32 * s;
    key[s] = e < N ? key_of(fmaf(unit, sc[s], bias ? __ldg(bias + e) : 0.0f)) : 0u;
  }

  if (groups > 1) {
    // lane g: the two best of group g, then its rank among the groups
    const int size = N / groups;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) s_key[lane + 32 * s] = key[s];
    __syncwarp();
    uint32_t gkey = 0;
    if (lane < groups) {
      uint32_t a = 0, b = 0;
      for (int i = 0; i < size; ++i) {
        const uint32_t q = s_key[lane * size + i];
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
      for (unsigned m = mask[s]; m != 0u; m &= m - 1u) sum += unit * __shfl_sync(kAll, sc[s], __ffs(m) - 1);
  }
  const float div = renormalize ? sum + 1e-20f : 1.0f;
  int base = 0;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    if ((chosen >> s) & 1u) {
      const int slot = base + __popc(mask[s] & ((1u << lane) - 1u));
      idx_out[slot] = lane + 32 * s;
      gate_out[slot] = scale * (unit * sc[s] / div);
    }
    base += __popc(mask[s]);
  }
}

__device__ __forceinline__ void order(float& a, float& b) {   // a >= b
  const float x = fmaxf(a, b);
  b = fminf(a, b);
  a = x;
}
__device__ __forceinline__ void sort4(float& a, float& b, float& c, float& d) {
  order(a, b);
  order(c, d);
  order(a, c);
  order(b, d);
  order(b, c);
}

// The four largest of a lane's E values, descending.
template <int E>
__device__ __forceinline__ void best_four(const float (&v)[E], float (&top)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) top[i] = v[i];
  sort4(top[0], top[1], top[2], top[3]);
#pragma unroll
  for (int g = 1; g < E / 4; ++g) {
    float o[4] = {v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
    sort4(o[0], o[1], o[2], o[3]);
    // the larger of top[i] and o[3 - i] are the four largest, a bitonic sequence
#pragma unroll
    for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], o[3 - i]);
    order(top[0], top[2]);
    order(top[1], top[3]);
    order(top[0], top[1]);
    order(top[2], top[3]);
  }
}

// Bits of a lane's `count` largest values, the last of them `last` (equal
// values: the lower index first); +inf and 0: none.
template <int E>
__device__ __forceinline__ uint32_t taken(const float (&v)[E], int count, float last) {
  uint32_t bits = 0;
#pragma unroll
  for (int s = 0; s < E; ++s) bits |= v[s] >= last ? 1u << s : 0u;
  if (__any_sync(0xffffffffu, __popc(bits) != count)) {   // more equal values than taken
    int equal = count;
#pragma unroll
    for (int s = 0; s < E; ++s) equal -= v[s] > last ? 1 : 0;
#pragma unroll
    for (int s = 0; s < E; ++s) {
      if (v[s] == last && --equal < 0) bits &= ~(1u << s);
    }
  }
  return bits;
}

// E consecutive experts a lane, W lanes a token; groups of 2^lanes_log2 lanes.
// -inf is "not available": a token with a NaN or +inf value, or with -inf among
// its k best, is left to route_row, which ranks every float.
template <int W, int E>
__global__ void __launch_bounds__(32 * kRouteWarps) route_lanes_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias, int T, int N, int k, int sigmoids, int groups,
    int lanes_log2, int top_groups, int top2, int renormalize, float scale, int32_t* __restrict__ idx_out,
    float* __restrict__ gate_out) {
  __shared__ uint32_t s_key[kRouteWarps][32 * kSlots];
  constexpr int kTokens = 32 / W;   // of a warp
  constexpr uint32_t kAll = 0xffffffffu;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % W, me = lane / W;
  const uint32_t mine = W == 32 ? kAll : ((1u << (W % 32)) - 1u) << (me * W);   // the token's lanes
  const uint32_t before = mine & ((1u << lane) - 1u);                            // those before this one
  const long long t0 = ((long long)blockIdx.x * kRouteWarps + warp) * kTokens;
  const long long t = t0 + me;
  pdl_wait();
  pdl_trigger();
  if (t0 >= T) return;
  const bool in = l * E < N && t < T;   // N % E == 0: a lane's experts exist or do not together
  float sc[E], b[E];
#pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    const float4 v = in ? __ldcs(reinterpret_cast<const float4*>(logits + t * N + l * E) + q)
                        : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    sc[4 * q] = v.x;
    sc[4 * q + 1] = v.y;
    sc[4 * q + 2] = v.z;
    sc[4 * q + 3] = v.w;
  }
  scores_of<W, E>(sc, sigmoids);
  const float unit = score_unit(sigmoids);
  float check = 0.0f;   // NaN or +inf if a value is; -inf values alone leave it -inf
#pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    const float4 v = bias && in ? __ldg(reinterpret_cast<const float4*>(bias + l * E) + q)
                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    b[4 * q] = fmaf(unit, sc[4 * q], v.x);
    b[4 * q + 1] = fmaf(unit, sc[4 * q + 1], v.y);
    b[4 * q + 2] = fmaf(unit, sc[4 * q + 2], v.z);
    b[4 * q + 3] = fmaf(unit, sc[4 * q + 3], v.w);
    check += b[4 * q] + b[4 * q + 1] + b[4 * q + 2] + b[4 * q + 3];
  }
  unsigned odd = __ballot_sync(kAll, !(check < INFINITY));
  float top[4];
  best_four<E>(b, top);
  if (!in) top[0] = top[1] = top[2] = top[3] = -INFINITY;

  if (groups > 1) {
    const int lanes = 1 << lanes_log2;   // of one group
    float x = top[0], y = top[1];
    for (int off = 1; off < lanes; off <<= 1) {
      const float ox = __shfl_xor_sync(kAll, x, off), oy = __shfl_xor_sync(kAll, y, off);
      y = fmaxf(fminf(x, ox), fmaxf(y, oy));
      x = fmaxf(x, ox);
    }
    // the group's rank: its lanes share the comparisons with the other groups
    const float score = top2 ? x + y : x;
    const int group = l >> lanes_log2;
    int better = 0;
    for (int g0 = 0; g0 < groups; g0 += lanes) {
      const int g = g0 + (l & (lanes - 1));
      const float o = __shfl_sync(kAll, score, me * W + ((g << lanes_log2) & (W - 1)));
      better += g < groups && (o > score || (o == score && g < group)) ? 1 : 0;
    }
    for (int off = 1; off < lanes; off <<= 1) better += __shfl_xor_sync(kAll, better, off);
    if (better >= top_groups) top[0] = top[1] = top[2] = top[3] = -INFINITY;
  }

  uint32_t chosen = 0;          // bit s: expert l * E + s is selected
  float last = INFINITY;        // the last value this lane gave up
  int count = 0;
  float best = 0.0f;
  for (int j = 0; j < k; ++j) {
    best = top[0];
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) best = fmaxf(best, __shfl_xor_sync(kAll, best, off));
    const bool eq = top[0] == best;
    const unsigned who = __ballot_sync(kAll, eq);
    if (eq && (who & before) == 0u) {   // the lowest lane: the lowest expert of equal values
      ++count;
      last = best;
      top[0] = top[1];
      top[1] = top[2];
      top[2] = top[3];
      top[3] = -INFINITY;
    }
    if (E > 4 && j >= 3 && __any_sync(kAll, count == 4)) {
      // a lane's list has run out: what it gave leaves its values, and the next four come
      const bool out = count == 4;
      const uint32_t bits = taken<E>(b, out ? 4 : 0, out ? last : INFINITY);
      chosen |= bits;
#pragma unroll
      for (int s = 0; s < E; ++s) b[s] = (bits >> s) & 1u ? -INFINITY : b[s];
      if (out) {
        best_four<E>(b, top);
        count = 0;
        last = INFINITY;
      }
    }
  }
  chosen |= taken<E>(b, count, last);
  // a token with such a value, or with fewer than k values above -inf (the last round found none),
  // has gone through the motions and is routed below
  odd |= __ballot_sync(kAll, best == -INFINITY && t < T);
  const bool left = (odd & mine) != 0u;
  if (left) chosen = 0u;

  // slots: the selected experts of the lanes before come first
  const int n = __popc(chosen);
  int slot = 0;
#pragma unroll
  for (int bit = 0; bit < 5; ++bit) slot += __popc(__ballot_sync(kAll, (n >> bit) & 1) & before) << bit;
  uint2* s_out = reinterpret_cast<uint2*>(s_key[warp]) + me * 16;   // k <= 16 slots a token
  uint2* out = s_out + slot;
#pragma unroll
  for (int s = 0; s < E; ++s)
    if ((chosen >> s) & 1u) *out++ = make_uint2(l * E + s, __float_as_uint(sc[s]));
  __syncwarp();
  const uint2 got = l < k ? s_out[l] : make_uint2(0, 0);
  float gate = unit * __uint_as_float(got.y), sum = gate;
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);   // the 16 slots
  gate = scale * (renormalize ? gate / (sum + 1e-20f) : gate);
  if (l < k && t < T && !left) {
    idx_out[t * k + l] = (int32_t)got.x;
    gate_out[t * k + l] = gate;
  }
  if (odd != 0u) {
    for (int i = 0; i < kTokens; ++i) {
      if (!(odd >> (i * W) & (kAll >> (32 - W)))) continue;
      __syncwarp();
      route_row(logits + (t0 + i) * N, bias, N, k, sigmoids, groups, top_groups, top2, renormalize, scale,
                s_key[warp], idx_out + (t0 + i) * k, gate_out + (t0 + i) * k);
    }
  }
}

__global__ void __launch_bounds__(32 * kRouteWarps) route_scored_kernel(
    const float* __restrict__ logits, const float* __restrict__ bias, int T, int N, int k, int sigmoids, int groups,
    int top_groups, int top2, int renormalize, float scale, int32_t* __restrict__ idx_out,
    float* __restrict__ gate_out) {
  __shared__ uint32_t s_key[kRouteWarps][32 * kSlots];
  const int warp = threadIdx.x >> 5;
  const long long t = (long long)blockIdx.x * kRouteWarps + warp;
  pdl_wait();
  pdl_trigger();
  if (t >= T) return;
  route_row(logits + t * N, bias, N, k, sigmoids, groups, top_groups, top2, renormalize, scale, s_key[warp],
            idx_out + t * k, gate_out + t * k);
}

}  // namespace

int route_scored_max_groups() { return kMaxGroups; }

void launch_route_scored(const float* logits, const float* bias, int T, int N, int k, bool sigmoid, int groups,
                         int top_groups, bool top2, bool renormalize, float scale, int32_t* topk_idx,
                         float* topk_gate, cudaStream_t s) {
  // a lane's experts lie in one group, and a group is a power of two of lanes
  auto lanes_ok = [&](int w, int e) {
    if (N % e || N > w * e) return false;
    if (groups == 1) return true;
    const int size = N / groups;
    return size % e == 0 && (size / e & (size / e - 1)) == 0;
  };
  auto go = [&](auto kernel, int w, int e) {
    const int tokens = kRouteWarps * (32 / w);
    int log2 = 0;
    while (groups > 1 && e << log2 < N / groups) ++log2;
    launch_pdl(kernel, dim3((T + tokens - 1) / tokens), dim3(32 * kRouteWarps), 0, s, logits, bias, T, N, k,
               sigmoid ? 1 : 0, groups, log2, top_groups, top2 ? 1 : 0, renormalize ? 1 : 0, scale, topk_idx,
               topk_gate);
  };
  if (lanes_ok(16, 4)) return go(route_lanes_kernel<16, 4>, 16, 4);
  if (lanes_ok(16, 8)) return go(route_lanes_kernel<16, 8>, 16, 8);
  if (lanes_ok(16, 16)) return go(route_lanes_kernel<16, 16>, 16, 16);
  if (lanes_ok(32, 4)) return go(route_lanes_kernel<32, 4>, 32, 4);
  if (lanes_ok(32, 8)) return go(route_lanes_kernel<32, 8>, 32, 8);
  const dim3 grid((T + kRouteWarps - 1) / kRouteWarps), block(32 * kRouteWarps);
  launch_pdl(route_scored_kernel, grid, block, 0, s, logits, bias, T, N, k, sigmoid ? 1 : 0,
             groups, top_groups, top2 ? 1 : 0, renormalize ? 1 : 0, scale, topk_idx, topk_gate);
}

}  // namespace moe
