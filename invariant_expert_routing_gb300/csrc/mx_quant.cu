// Conversion between bf16 and the microscaled 4-bit format (mx.cuh): rows,
// weights stored [experts, K, features] (blocks run along K, so this one
// transposes), back to bf16, and the scale layout of the grouped GEMM.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "kernels.h"
#include "mx.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

using namespace mx;

// Rows to codes and scales: four lanes a block, eight elements (16 bytes
// read, 4 written) a lane, four such pieces in flight.  Bound by memory (2.53
// bytes an element): 16448 x 7168 elements here and back through
// dequantize_kernel, 597 MB, in 91 us (6.6 TB/s; a plain copy runs at 6.8).
constexpr int kQuantThreads = 256;
constexpr int kQuantUnroll = 4;

__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const uint4* __restrict__ x, size_t n8,
                                                                      uint32_t* __restrict__ codes,
                                                                      uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const size_t base = (size_t)blockIdx.x * (kQuantThreads * kQuantUnroll) + threadIdx.x;
  uint4 v[kQuantUnroll];
#pragma unroll
  for (int u = 0; u < kQuantUnroll; ++u) {
    const size_t i = base + (size_t)u * kQuantThreads;
    v[u] = i < n8 ? __ldg(x + i) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < kQuantUnroll; ++u) {
    const size_t i = base + (size_t)u * kQuantThreads;
    uint32_t byte;
    const uint32_t c = quantize8(v[u], byte);
    if (i < n8) {
      codes[i] = c;
      if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
    }
  }
}

// Codes and scales back to bf16: eight elements a thread.
__global__ void __launch_bounds__(kQuantThreads) dequantize_kernel(const uint32_t* __restrict__ codes,
                                                                   const uint8_t* __restrict__ scales, size_t n8,
                                                                   uint4* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const size_t base = (size_t)blockIdx.x * (kQuantThreads * kQuantUnroll) + threadIdx.x;
  uint32_t c[kQuantUnroll], b[kQuantUnroll];
#pragma unroll
  for (int u = 0; u < kQuantUnroll; ++u) {
    const size_t i = base + (size_t)u * kQuantThreads;
    c[u] = i < n8 ? __ldg(codes + i) : 0u;
    b[u] = i < n8 ? __ldg(scales + (i >> 2)) : 0u;
  }
#pragma unroll
  for (int u = 0; u < kQuantUnroll; ++u) {
    const size_t i = base + (size_t)u * kQuantThreads;
    if (i >= n8) continue;
    uint32_t h[4], r[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c[u]));
    const float s = scale_value(b[u]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
      const __nv_bfloat162 p = __floats2bfloat162_rn(f.x * s, f.y * s);
      r[j] = *reinterpret_cast<const uint32_t*>(&p);
    }
    out[i] = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

// Weights [K, F] of one expert to codes [F, K/2] and scales [F, K/32].  A CTA
// takes 256 K x 64 features: each warp one block of 32 K, a lane two
// neighbouring features (32 loads of 4 bytes, 128 contiguous bytes a warp);
// the codes pass through shared memory so that each feature's 128 bytes leave
// as whole sectors.  Bound by memory: 128 x 2048 x 1536 elements here and back
// through dequantize_kernel, 2.04 GB, in 297 us (6.9 TB/s).
constexpr int kWqK = 256, kWqF = 64;

__global__ void __launch_bounds__(256) quantize_weights_kernel(const uint32_t* __restrict__ w, int K, int F,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
  __shared__ uint4 s_codes[kWqF][kWqK / 32 + 1];
  __shared__ uint8_t s_scales[kWqF][kWqK / 32];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k0 = (int)blockIdx.x * kWqK, f0 = (int)blockIdx.y * kWqF;
  const size_t e = blockIdx.z;
  const int kb = k0 + warp * kBlock, f = f0 + 2 * lane;
  if (kb < K && f < F) {   // F is even
    const uint32_t* src = w + ((e * K + kb) * F + f) / 2;
    const size_t ld = (size_t)F / 2;
    uint32_t v[kBlock];
#pragma unroll
    for (int i = 0; i < kBlock; ++i) v[i] = __ldg(src + i * ld);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kBlock; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t byte = scale_byte(half ? m & 0xFFFF0000u : m << 16);
      uint32_t c[4] = {0, 0, 0, 0};
      if (byte != 255u) {
        const float inv = scale_inverse(byte);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float t[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t x = v[8 * q + i];
            t[i] = __uint_as_float(half ? x & 0xFFFF0000u : x << 16) * inv;
          }
          c[q] = pack8(t);
        }
      }
      s_codes[2 * lane + half][warp] = make_uint4(c[0], c[1], c[2], c[3]);
      s_scales[2 * lane + half][warp] = (uint8_t)byte;
    }
  }
  __syncthreads();
  const int blocks = min(kWqK, K - k0) / kBlock;
  for (int i = threadIdx.x; i < kWqF * (kWqK / kBlock); i += blockDim.x) {
    const int fl = i / (kWqK / kBlock), b = i % (kWqK / kBlock);
    if (b < blocks && f0 + fl < F) {
      const size_t row = e * F + f0 + fl;
      *reinterpret_cast<uint4*>(codes + row * (K / 2) + k0 / 2 + 16 * b) = s_codes[fl][b];
      scales[row * (K / kBlock) + k0 / kBlock + b] = s_scales[fl][b];
    }
  }
}

// Scales [rows, K/32] of one expert into chunks of 128 rows x 128 K (four
// bytes a row, placed by sf_row_offset), chunks of a row tile contiguous
// along K.  gate_up: the rows are I gate rows then I up rows, and tile row r
// takes, in turns of 32, gate features and the same up features, the order
// in which the W13 GEMM reads them.  Run once for a set of weights; reads are
// four bytes K/32 apart, from L2 after the first of a row.
__global__ void __launch_bounds__(256) pack_scales_kernel(const uint32_t* __restrict__ scales, int rows, int kchunks,
                                                          int gate_up, uint32_t* __restrict__ out, size_t total) {
  pdl_wait();
  pdl_trigger();
  const size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x;   // one 4-byte word of the output
  if (i >= total) return;
  const int word = (int)(i % (kSfChunkBytes / 4));
  const size_t chunk = i / (kSfChunkBytes / 4);
  const int kc = (int)(chunk % kchunks);
  const size_t tile = chunk / kchunks;                 // over experts and row tiles
  const int tiles = rows / kSfRows;
  const size_t e = tile / tiles;
  const int r = (word & 3) * 32 + (word >> 2);          // row of the chunk
  int row = (int)(tile % tiles) * kSfRows + r;
  if (gate_up) {
    const int group = row >> 6, in = row & 63;          // 64 tile rows: 32 gate, 32 up features
    row = (in >> 5) * (rows / 2) + group * 32 + (in & 31);
  }
  out[i] = __ldg(scales + (e * rows + row) * kchunks + kc);
}

}  // namespace

void launch_quantize_mx(const uint16_t* x, size_t elements, uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  const size_t n8 = elements / 8;
  const size_t per = (size_t)kQuantThreads * kQuantUnroll;
  launch_pdl(quantize_rows_kernel, dim3((unsigned)((n8 + per - 1) / per)), dim3(kQuantThreads), 0, s,
             reinterpret_cast<const uint4*>(x), n8, reinterpret_cast<uint32_t*>(codes), scales);
}

void launch_dequantize_mx(const uint8_t* codes, const uint8_t* scales, size_t elements, uint16_t* out,
                          cudaStream_t s) {
  const size_t n8 = elements / 8;
  const size_t per = (size_t)kQuantThreads * kQuantUnroll;
  launch_pdl(dequantize_kernel, dim3((unsigned)((n8 + per - 1) / per)), dim3(kQuantThreads), 0, s,
             reinterpret_cast<const uint32_t*>(codes), scales, n8, reinterpret_cast<uint4*>(out));
}

void launch_quantize_weights_mx(const uint16_t* w, int experts, int K, int F, uint8_t* codes, uint8_t* scales,
                                cudaStream_t s) {
  launch_pdl(quantize_weights_kernel, dim3((K + kWqK - 1) / kWqK, (F + kWqF - 1) / kWqF, experts), dim3(256), 0, s,
             reinterpret_cast<const uint32_t*>(w), K, F, codes, scales);
}

void launch_pack_scales_mx(const uint8_t* scales, int experts, int rows, int K, bool gate_up, uint8_t* packed,
                           cudaStream_t s) {
  const size_t total = (size_t)experts * rows * (K / kBlock) / 4;
  launch_pdl(pack_scales_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s,
             reinterpret_cast<const uint32_t*>(scales), rows, K / kSfChunkK, gate_up ? 1 : 0,
             reinterpret_cast<uint32_t*>(packed), total);
}

}  // namespace moe
