// Products grouped by expert (ragged row counts) and the weight gradient:
//   y[p] = x[row(p)] . W_e      (or . W_e^T)          for every row p of expert e
//   dW_e = sum over its rows of x[row(p)]^T dy[row(p)]  (+ add_e)
// row(p) is p, or for a gathered operand the token of route ids[p].
//
// 64 x 64 tiles of fp32 sums on the CUDA cores, one K order for every batch.
#include <cuda_bf16.h>
#include <cstdint>

#include "gemm.h"
#include "grouped.h"
#include "kernels.h"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kMaxExperts = 256;
constexpr int kTile = 64, kStep = 16;

struct Segments {
  int start[kMaxExperts], count[kMaxExperts], first[kMaxExperts + 1];   // first: tiles before the expert's
  int ok;
};

// Segment starts and tile numbers from the experts' counts; every thread of
// the CTA calls it.  ok: the counts fit into max_rows rows.
__device__ void find_segments(const GroupArgs& a, int tile_rows, Segments& s) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    long long row = 0;
    int tile = 0, bad = 0;
    for (int e0 = 0; e0 < a.N; e0 += 32) {
      const int e = e0 + lane;
      const int c = e < a.N ? a.counts[e] : 0;
      bad |= c < 0 || c > a.max_rows;
      const long long padded = bad ? 0 : ((long long)c + a.B - 1) / a.B * a.B;
      const int tiles = bad ? 0 : (c + tile_rows - 1) / tile_rows;
      long long r = padded;
      int t = tiles;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long long ru = __shfl_up_sync(0xffffffffu, r, off);
        const int tu = __shfl_up_sync(0xffffffffu, t, off);
        if (lane >= off) r += ru, t += tu;
      }
      if (e < a.N) {
        s.start[e] = (int)(row + r - padded);
        s.count[e] = c;
        s.first[e] = tile + t - tiles;
      }
      row += __shfl_sync(0xffffffffu, r, 31);
      tile += __shfl_sync(0xffffffffu, t, 31);
    }
    bad |= row > a.max_rows;
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      s.first[a.N] = tile;
      s.ok = !bad;
      if (bad) atomicOr(a.status, kDevErrBadBlocks);
    }
  }
  __syncthreads();
}

// Row of the operand that grouped row p reads, -1: zeros.
__device__ __forceinline__ long long source_row(const GroupArgs& a, int gather, long long p) {
  if (!gather) return p;
  const int r = a.ids[p];
  return r >= 0 && r < a.T * a.slots ? r / a.slots : -1;
}
__device__ __forceinline__ float bf16_at(const uint16_t* p, size_t i) { return __uint_as_float((uint32_t)p[i] << 16); }

// acc[i][j] += sum over kk of a[kk][4 ty + i] * b[kk][4 tx + j]
__device__ __forceinline__ void tile_fma(const float (*a)[kTile + 4], const float (*b)[kTile + 4], float (&acc)[4][4]) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
#pragma unroll
  for (int kk = 0; kk < kStep; ++kk) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[kk][4 * ty + i], b[kk][4 * tx + j], acc[i][j]);
  }
}

__global__ void __launch_bounds__(256) grouped_gemm_kernel(const GroupedGemmArgs a) {
  __shared__ Segments seg;
  __shared__ float sx[kStep][kTile + 4], sw[kStep][kTile + 4];
  __shared__ long long s_row[kTile];
  pdl_wait();
  pdl_trigger();
  const GroupArgs& g = a.g;
  find_segments(g, kTile, seg);
  const int tile = blockIdx.x;
  if (!seg.ok || tile >= seg.first[g.N]) return;
  int e = 0;
  while (seg.first[e + 1] <= tile) ++e;
  const int r0 = (tile - seg.first[e]) * kTile, rows = min(kTile, seg.count[e] - r0), f0 = blockIdx.y * kTile;
  const long long p0 = seg.start[e] + r0;
  if (threadIdx.x < kTile) s_row[threadIdx.x] = (int)threadIdx.x < rows ? source_row(g, a.gather, p0 + threadIdx.x) : -1;
  __syncthreads();
  const uint16_t* w = a.w + (size_t)e * g.K * g.F;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += kStep) {
    for (int i = threadIdx.x; i < kStep * kTile; i += 256) {
      const int kk = i % kStep, m = i / kStep;
      const long long r = s_row[m];
      sx[kk][m] = r >= 0 && k0 + kk < g.K ? bf16_at(a.x, (size_t)r * g.K + k0 + kk) : 0.0f;
      const int wk = a.transposed ? kk : i / kTile, n = a.transposed ? m : i % kTile;
      const bool in = k0 + wk < g.K && f0 + n < g.F;
      sw[wk][n] = !in ? 0.0f
                      : bf16_at(w, a.transposed ? (size_t)(f0 + n) * g.K + k0 + wk : (size_t)(k0 + wk) * g.F + f0 + n);
    }
    __syncthreads();
    tile_fma(sx, sw, acc);
    __syncthreads();
  }
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = 4 * ty + i, n = f0 + 4 * tx + j;
      if (m < rows && n < g.F)
        reinterpret_cast<__nv_bfloat16*>(a.y)[(size_t)(p0 + m) * g.F + n] = __float2bfloat16_rn(acc[i][j]);
    }
}

__global__ void __launch_bounds__(256) grouped_wgrad_kernel(const GroupedWgradArgs a) {
  __shared__ Segments seg;
  __shared__ float sx[kStep][kTile + 4], sd[kStep][kTile + 4];
  pdl_wait();
  pdl_trigger();
  const GroupArgs& g = a.g;
  find_segments(g, kTile, seg);
  if (!seg.ok) return;
  const int e = blockIdx.z, k0 = blockIdx.y * kTile, f0 = blockIdx.x * kTile, rows = seg.count[e];
  const long long p0 = seg.start[e];
  float acc[4][4] = {};
  for (int r0 = 0; r0 < rows; r0 += kStep) {
    for (int i = threadIdx.x; i < kStep * kTile; i += 256) {
      const int rr = i / kTile, c = i % kTile;
      const bool in = r0 + rr < rows;
      const long long rx = in ? source_row(g, a.gather_x, p0 + r0 + rr) : -1;
      const long long rd = in ? source_row(g, a.gather_dy, p0 + r0 + rr) : -1;
      sx[rr][c] = rx >= 0 && k0 + c < g.K ? bf16_at(a.x, (size_t)rx * g.K + k0 + c) : 0.0f;
      sd[rr][c] = rd >= 0 && f0 + c < g.F ? bf16_at(a.dy, (size_t)rd * g.F + f0 + c) : 0.0f;
    }
    __syncthreads();
    tile_fma(sx, sd, acc);
    __syncthreads();
  }
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = k0 + 4 * ty + i, n = f0 + 4 * tx + j;
      if (m >= g.K || n >= g.F) continue;
      const size_t at = ((size_t)e * g.K + m) * g.F + n;
      if (!a.fp32)
        reinterpret_cast<__nv_bfloat16*>(a.dw)[at] = __float2bfloat16_rn(acc[i][j]);
      else
        reinterpret_cast<float*>(a.dw)[at] = a.add ? a.add[at] + acc[i][j] : acc[i][j];
    }
}

}  // namespace

void launch_grouped_gemm(const GroupedGemmArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)(a.g.max_rows / kTile + a.g.N), (a.g.F + kTile - 1) / kTile);
  launch_pdl(grouped_gemm_kernel, grid, dim3(256), 0, s, a);
}

void launch_grouped_wgrad(const GroupedWgradArgs& a, cudaStream_t s) {
  const dim3 grid((a.g.F + kTile - 1) / kTile, (a.g.K + kTile - 1) / kTile, a.g.N);
  launch_pdl(grouped_wgrad_kernel, grid, dim3(256), 0, s, a);
}

}  // namespace moe
