// Residual addition and root-mean-square norm, with the normalised row also
// in microscaled 4 bits:
//   v = x + residual (fp32);  residual_out = bf16(v)
//   out = bf16(v / sqrt(mean(v^2) + eps) * weight);  codes, scales = MX e2m1 of out
// One CTA a row, the row in registers between the two passes, so each byte
// moves once: bound by memory (8 bytes an element, 0.53 more with the codes).
// 16448 rows of 7168 with codes, then the codes back to bf16, 1.30 GB, take
// 193 us (6.8 TB/s, the rate of a plain copy); one row 2 us on the device.
//
// The sum of squares has one order for every batch and thread count: eight
// elements in turn, the 32 groups of a 256-element chunk by a fixed tree,
// then the chunks by another.  How many warps share a row is thus
// free to follow the batch.
#include <cuda_bf16.h>
#include <cstdint>

#include "bf16x8.cuh"
#include "kernels.h"
#include "mx.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kNormChunk = 256;      // elements a warp takes at once (eight a lane)
constexpr int kNormMaxChunks = 128;  // H <= 32768

// NV: 256-element chunks a warp holds.  residual_out and out may be x or
// residual (no __restrict__ on the four): a row is read before the barrier and
// written after it.
template <int NV>
__global__ void __launch_bounds__(1024) add_norm_kernel(const uint16_t* x, const uint16_t* residual,
                                                        const uint16_t* __restrict__ weight, float eps, int H,
                                                        uint16_t* residual_out, uint16_t* out,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ float s_sum[kNormMaxChunks];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int chunks = (H + kNormChunk - 1) / kNormChunk;
  const size_t row = (size_t)blockIdx.x * H;
  pdl_wait();
  pdl_trigger();
  uint4 xv[NV], rv[NV], wv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (warp + i * warps) * kNormChunk + lane * 8;
    const bool in = c < H;
    xv[i] = in ? __ldcs(reinterpret_cast<const uint4*>(x + row + c)) : make_uint4(0, 0, 0, 0);
    rv[i] = in && residual ? __ldcs(reinterpret_cast<const uint4*>(residual + row + c)) : make_uint4(0, 0, 0, 0);
    wv[i] = in ? __ldg(reinterpret_cast<const uint4*>(weight + c)) : make_uint4(0, 0, 0, 0);
  }
  float v[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float r[8];
    unpack8(xv[i], v[i]);
    unpack8(rv[i], r);
    float q = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (residual) v[i][j] += r[j];
      q = fmaf(v[i][j], v[i][j], q);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) q += __shfl_xor_sync(0xffffffffu, q, off);
    const int c = warp + i * warps;
    if (lane == 0 && c < chunks) s_sum[c] = q;
  }
  __syncthreads();
  float total = 0.0f;
#pragma unroll
  for (int c = 0; c < kNormMaxChunks; c += 64) {
    float u = c + lane < chunks ? s_sum[c + lane] : 0.0f;
    if (c + 32 + lane < chunks) u += s_sum[c + 32 + lane];
    total += u;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  const float root = sqrtf(total / (float)H + eps), inv = 1.0f / root;
  const bool normal = root > 0.0f && root <= 3.402823466e38f;   // no correction of a quotient by zero or infinity
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (warp + i * warps) * kNormChunk + lane * 8;
    const bool in = c < H;
    if (in && residual_out) __stcs(reinterpret_cast<uint4*>(residual_out + row + c), pack_bf16(v[i]));
    float w[8], n[8];
    unpack8(wv[i], w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // v / root with one correction: the product alone rounds twice, which
      // turns a bf16 rounding (and a 4-bit one behind it) twice as often
      const float q = v[i][j] * inv;
      n[j] = (normal ? fmaf(fmaf(-q, root, v[i][j]), inv, q) : q) * w[j];
    }
    const uint4 nb = pack_bf16(n);
    if (in && out) *reinterpret_cast<uint4*>(out + row + c) = nb;
    if (codes) {
      uint32_t byte;
      const uint32_t q = mx::quantize8(nb, byte);
      if (in) {
        *reinterpret_cast<uint32_t*>(codes + (row + c) / 2) = q;
        if ((lane & 3) == 0) scales[(row + c) / mx::kBlock] = (uint8_t)byte;
      }
    }
  }
}

}  // namespace

void launch_add_norm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps, int T, int H,
                     uint16_t* residual_out, uint16_t* out, uint8_t* codes, uint8_t* scales, int sms,
                     cudaStream_t s) {
  const int chunks = (H + kNormChunk - 1) / kNormChunk;
  // few rows: one chunk a warp, for the shortest path; many: four, so that an
  // SM holds several rows and their loads overlap
  int nv = T < 4 * sms && chunks <= 32 ? 1 : 4;
  const int warps = (chunks + nv - 1) / nv;
  const dim3 grid((unsigned)T), block(32 * warps);
  auto go = [&](auto kernel) {
    launch_pdl(kernel, grid, block, 0, s, x, residual, weight, eps, H, residual_out, out, codes, scales);
  };
  if (nv == 1)
    go(add_norm_kernel<1>);
  else
    go(add_norm_kernel<4>);
}

}  // namespace moe
