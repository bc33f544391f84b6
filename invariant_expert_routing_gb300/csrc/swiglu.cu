// The activation between the two expert products, with the routes' gates, and
// its gradient, over grouped rows:
//   a = w silu(g) u           g, u = the halves of a row of gu [rows, 2I]
//   dg = w da u s (1 + g (1 - s)),  du = w da silu(g),  s = 1 / (1 + e^-g)
//   dw = sum over I of da silu(g) u
// w is the gate of the row's route (1 without gates).  Memory bound: 6 bytes an
// element of a forward, 10 backward, 12 with a written again.
//
// Forward: eight elements a thread at a time, any row's (rows are not shared out
// to CTAs: a row of 768 would leave most of a CTA idle).  Backward: one CTA a
// row, since dw is summed in one order for every batch (a thread's elements in
// turn, its warp's lanes by a fixed tree, then the warps in turn; the threads
// follow I alone).  4096 tokens of the 8-expert layer backward, 1.41 GB: 210 us
// (6.7 TB/s, the rate of a plain copy); 512 tokens of the 128-expert layer
// forward, 19 MB: 4.1 us (a CTA a row: 6.5).  Short rows backward, 65536 of them: of
// 768 96 us for 89 by the bytes, of 128 (one warp a CTA) 69 for 15: the CTAs bound.  A
// CTA is launched for every row that could be: one token, 256 experts and blocks of
// 128 rows are 32520 CTAs for 8 rows, 33 us.
//
// The sigmoid is the fast exponential and division, off by (6 + 1.2 |g|) 2^-23 at
// most: far below the bf16 roundings of a and dgu, and dgate's stated bound.
#include <cuda_bf16.h>
#include <cstdint>

#include "bf16x8.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kSwigluThreads = 256;

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// Thread (piece of 8 columns, row group): consecutive threads take consecutive
// pieces of a row, then of the next one.
__global__ void __launch_bounds__(kSwigluThreads)
    swiglu_kernel(const uint16_t* __restrict__ gu, const float* __restrict__ gates, const int32_t* __restrict__ ids,
                  const int32_t* __restrict__ num_padded, long long max_rows, int R, int I, uint16_t* __restrict__ a) {
  pdl_wait();
  pdl_trigger();
  const long long P = min((long long)*num_padded, max_rows);
  const int pieces = I / 8;
  const long long n = P * pieces, step = (long long)gridDim.x * blockDim.x;
  for (long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x; at < n; at += step) {
    const long long p = at / pieces;
    const int c = (int)(at - p * pieces) * 8, r = __ldg(ids + p);
    if (r < 0 || r >= R) continue;
    const size_t row = (size_t)p * I + c, row2 = 2 * (size_t)p * I + c;
    float g[8], u[8], o[8];
    unpack8(__ldcs(reinterpret_cast<const uint4*>(gu + row2)), g);
    unpack8(__ldcs(reinterpret_cast<const uint4*>(gu + row2 + I)), u);
    const float w = gates ? __ldg(gates + r) : 1.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = g[j] * sigmoid(g[j]) * (w * u[j]);
    *reinterpret_cast<uint4*>(a + row) = pack_bf16(o);
  }
}

// gu may be dgu and da may be a: each element is read before the same thread
// writes it (no __restrict__ on the four).
__global__ void __launch_bounds__(kSwigluThreads)
    swiglu_backward_kernel(const uint16_t* gu, const float* __restrict__ gates, const uint16_t* da,
                           const int32_t* __restrict__ ids, const int32_t* __restrict__ num_padded, long long max_rows,
                           int R, int I, uint16_t* a, uint16_t* dgu, float* __restrict__ dgate) {
  __shared__ float s_sum[kSwigluThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  const long long P = min((long long)*num_padded, max_rows);
  for (long long p = blockIdx.x; p < P; p += gridDim.x) {
    const int r = ids[p];
    if (r < 0 || r >= R) continue;   // the same for the whole CTA
    const float w = gates ? gates[r] : 1.0f;
    const size_t row = (size_t)p * I, row2 = 2 * row;
    float sum = 0.0f;
    for (int c = threadIdx.x * 8; c < I; c += blockDim.x * 8) {
      float g[8], u[8], d[8], o[8], og[8], ou[8];
      unpack8(__ldcs(reinterpret_cast<const uint4*>(gu + row2 + c)), g);
      unpack8(__ldcs(reinterpret_cast<const uint4*>(gu + row2 + I + c)), u);
      unpack8(__ldcs(reinterpret_cast<const uint4*>(da + row + c)), d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = sigmoid(g[j]);
        const float silu = g[j] * s, wu = w * u[j];
        o[j] = silu * wu;
        sum = fmaf(d[j], silu * u[j], sum);
        og[j] = d[j] * wu * (s * fmaf(g[j], 1.0f - s, 1.0f));
        ou[j] = w * d[j] * silu;
      }
      if (a) *reinterpret_cast<uint4*>(a + row + c) = pack_bf16(o);
      *reinterpret_cast<uint4*>(dgu + row2 + c) = pack_bf16(og);
      *reinterpret_cast<uint4*>(dgu + row2 + I + c) = pack_bf16(ou);
    }
    if (dgate) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      __syncthreads();   // the row before is done with s_sum
      if (lane == 0) s_sum[warp] = sum;
      __syncthreads();
      if (threadIdx.x == 0) {
        float t = 0.0f;
        for (int i = 0; i < (int)blockDim.x / 32; ++i) t += s_sum[i];
        dgate[r] = t;
      }
    }
  }
}

}  // namespace

void launch_swiglu(const uint16_t* gu, const float* gates, const int32_t* ids, const int32_t* num_padded,
                   int64_t max_rows, int R, int I, uint16_t* a, cudaStream_t s) {
  const int64_t ctas = (max_rows * (I / 8) + kSwigluThreads - 1) / kSwigluThreads, most = 152 * 8 * 4;
  launch_pdl(swiglu_kernel, dim3((unsigned)(ctas < most ? ctas : most)), dim3(kSwigluThreads), 0, s, gu, gates, ids,
             num_padded, (long long)max_rows, R, I, a);
}

void launch_swiglu_backward(const uint16_t* gu, const float* gates, const uint16_t* da, const int32_t* ids,
                            const int32_t* num_padded, int64_t max_rows, int R, int I, uint16_t* dgu, float* dgate,
                            uint16_t* a, cudaStream_t s) {
  const int want = (I / 8 + 31) / 32 * 32;
  const int threads = want < kSwigluThreads ? want : kSwigluThreads;
  const int64_t grid = max_rows < (1 << 20) ? max_rows : (1 << 20);
  launch_pdl(swiglu_backward_kernel, dim3((unsigned)grid), dim3(threads), 0, s, gu, gates, da, ids, num_padded,
             (long long)max_rows, R, I, a, dgu, dgate);
}

}  // namespace moe
