// Residual addition and layer norm, and the gradients of the layer norm and of
// the root-mean-square norm:
//   v = x + residual;  out = (v - mean) / sqrt(var + eps) * weight + bias
//   g = dout * weight;  n = (v - mean) / sqrt(var + eps)
//   dv = dresidual + (g - mean(g) - n mean(g n)) / sqrt(var + eps)
//   dweight = sum over rows of dout n;  dbias = sum over rows of dout
// (RMS norm: mean = 0, mean(g) left out).  The statistics are computed again
// from v: the row is read anyway.  Variances come from the deviations, so a
// mean far from zero costs no digits.
//
// Sums over a row have one order for every batch: eight elements in turn, the
// 32 groups of a 256-element chunk by a fixed tree, the chunks by another.
#include <cuda_bf16.h>
#include <cstdint>

#include "bf16x8.cuh"
#include "kernels.h"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kChunk = 256;       // elements a warp takes at once (eight a lane)
constexpr int kMaxChunks = 128;   // H <= 32768

// Sums of the row's chunks q[i] (chunk warp + i * warps), known to every thread.
// s_sum: one array a call, so that one barrier is enough.
template <int NV>
__device__ __forceinline__ float row_sum(float (&q)[NV], int warp, int warps, int lane, int chunks, float* s_sum) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) q[i] += __shfl_xor_sync(0xffffffffu, q[i], off);
    const int c = warp + i * warps;
    if (lane == 0 && c < chunks) s_sum[c] = q[i];
  }
  __syncthreads();
  float total = 0.0f;
#pragma unroll
  for (int c = 0; c < kMaxChunks; c += 64) {
    float u = c + lane < chunks ? s_sum[c + lane] : 0.0f;
    if (c + 32 + lane < chunks) u += s_sum[c + 32 + lane];
    total += u;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  return total;
}

// residual_out and out may be x or residual (no __restrict__ on the four): a
// row is read before the first barrier and written after it.
template <int NV>
__global__ void __launch_bounds__(1024)
    add_layer_norm_kernel(const uint16_t* x, const uint16_t* residual, const uint16_t* __restrict__ weight,
                          const uint16_t* __restrict__ bias, float eps, int H, uint16_t* residual_out, uint16_t* out) {
  __shared__ float s_sum[2][kMaxChunks];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int chunks = (H + kChunk - 1) / kChunk;
  const size_t row = (size_t)blockIdx.x * H;
  pdl_wait();
  pdl_trigger();
  uint4 xv[NV], rv[NV], wv[NV], bv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (warp + i * warps) * kChunk + lane * 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    xv[i] = c < H ? __ldcs(reinterpret_cast<const uint4*>(x + row + c)) : zero;
    rv[i] = c < H && residual ? __ldcs(reinterpret_cast<const uint4*>(residual + row + c)) : zero;
    wv[i] = c < H ? __ldg(reinterpret_cast<const uint4*>(weight + c)) : zero;
    bv[i] = c < H && bias ? __ldg(reinterpret_cast<const uint4*>(bias + c)) : zero;
  }
  float v[NV][8], q[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float r[8];
    unpack8(xv[i], v[i]);
    unpack8(rv[i], r);
    q[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (residual) v[i][j] += r[j];
      q[i] += v[i][j];
    }
  }
  const float mean = row_sum<NV>(q, warp, warps, lane, chunks, s_sum[0]) / (float)H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (warp + i * warps) * kChunk + lane * 8;
    if (c < H && residual_out) __stcs(reinterpret_cast<uint4*>(residual_out + row + c), pack_bf16(v[i]));
    q[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = c < H ? v[i][j] - mean : 0.0f;
      q[i] = fmaf(v[i][j], v[i][j], q[i]);
    }
  }
  const float var = row_sum<NV>(q, warp, warps, lane, chunks, s_sum[1]) / (float)H;
  const float inv = 1.0f / sqrtf(var + eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (warp + i * warps) * kChunk + lane * 8;
    float w[8], b[8];
    unpack8(wv[i], w);
    unpack8(bv[i], b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * inv, w[j], b[j]);
    if (c < H) *reinterpret_cast<uint4*>(out + row + c) = pack_bf16(v[i]);
  }
}

// dv of one row a CTA, and the row's (mean, 1 / root) for the weight's gradient.
// dx may be dresidual (no __restrict__): a row is read before the first barrier.
template <int NV>
__global__ void __launch_bounds__(1024)
    norm_dx_kernel(const uint16_t* v_in, const uint16_t* dout, const uint16_t* dresidual,
                   const uint16_t* __restrict__ weight, float eps, int H, int centre, uint16_t* dx, float2* stats) {
  __shared__ float s_sum[4][kMaxChunks];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int chunks = (H + kChunk - 1) / kChunk;
  const size_t row = (size_t)blockIdx.x * H;
  pdl_wait();
  pdl_trigger();
  uint4 vv[NV], gv[NV], rv[NV], wv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (warp + i * warps) * kChunk + lane * 8;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    vv[i] = c < H ? *reinterpret_cast<const uint4*>(v_in + row + c) : zero;
    gv[i] = c < H ? *reinterpret_cast<const uint4*>(dout + row + c) : zero;
    rv[i] = c < H && dresidual ? *reinterpret_cast<const uint4*>(dresidual + row + c) : zero;
    wv[i] = c < H ? __ldg(reinterpret_cast<const uint4*>(weight + c)) : zero;
  }
  float v[NV][8], g[NV][8], q[NV], p[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[8];
    unpack8(vv[i], v[i]);
    unpack8(gv[i], g[i]);
    unpack8(wv[i], w);
    q[i] = p[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[i][j] *= w[j];
      q[i] += v[i][j];
      p[i] += g[i][j];
    }
  }
  const float sv = row_sum<NV>(q, warp, warps, lane, chunks, s_sum[0]);
  const float sg = row_sum<NV>(p, warp, warps, lane, chunks, s_sum[1]);
  const float mean = centre ? sv / (float)H : 0.0f, mean_g = centre ? sg / (float)H : 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (warp + i * warps) * kChunk + lane * 8;
    q[i] = p[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] = c < H ? v[i][j] - mean : 0.0f;
      q[i] = fmaf(v[i][j], v[i][j], q[i]);
      p[i] = fmaf(v[i][j], g[i][j], p[i]);
    }
  }
  const float var = row_sum<NV>(q, warp, warps, lane, chunks, s_sum[2]) / (float)H;
  const float sgd = row_sum<NV>(p, warp, warps, lane, chunks, s_sum[3]);
  const float inv = 1.0f / sqrtf(var + eps);
  const float slope = sgd / (float)H * inv * inv;   // mean(g n) / root
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (warp + i * warps) * kChunk + lane * 8;
    float r[8];
    unpack8(rv[i], r);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = fmaf(g[i][j] - mean_g - v[i][j] * slope, inv, r[j]);
    if (c < H) *reinterpret_cast<uint4*>(dx + row + c) = pack_bf16(v[i]);
  }
  if (threadIdx.x == 0) stats[blockIdx.x] = make_float2(mean, inv);
}

// part[slab][0 / 1][H]: sums over the rows of a slab of dout n and dout.
__global__ void __launch_bounds__(128)
    norm_columns_kernel(const uint16_t* __restrict__ v_in, const uint16_t* __restrict__ dout,
                        const float2* __restrict__ stats, int T, int H, int slab_rows, float* __restrict__ part) {
  const int c = (blockIdx.x * 128 + threadIdx.x) * 2;
  pdl_wait();
  pdl_trigger();
  if (c >= H) return;
  const int t0 = blockIdx.y * slab_rows, t1 = min(T, t0 + slab_rows);
  float dw0 = 0.0f, dw1 = 0.0f, db0 = 0.0f, db1 = 0.0f;
  for (int t = t0; t < t1; ++t) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(v_in + (size_t)t * H + c);
    const uint32_t d = *reinterpret_cast<const uint32_t*>(dout + (size_t)t * H + c);
    const float2 s = stats[t];
    const float d0 = __uint_as_float(d << 16), d1 = __uint_as_float(d & 0xFFFF0000u);
    dw0 = fmaf(d0, (__uint_as_float(v << 16) - s.x) * s.y, dw0);
    dw1 = fmaf(d1, (__uint_as_float(v & 0xFFFF0000u) - s.x) * s.y, dw1);
    db0 += d0;
    db1 += d1;
  }
  float* at = part + (size_t)blockIdx.y * 2 * H + c;
  *reinterpret_cast<float2*>(at) = make_float2(dw0, dw1);
  *reinterpret_cast<float2*>(at + H) = make_float2(db0, db1);
}

__global__ void __launch_bounds__(128)
    norm_columns_sum_kernel(const float* __restrict__ part, int slabs, int H, float* __restrict__ dweight,
                            float* __restrict__ dbias) {
  const int c = blockIdx.x * 128 + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (c >= H) return;
  float dw = 0.0f, db = 0.0f;
  for (int s = 0; s < slabs; ++s) {
    dw += part[(size_t)s * 2 * H + c];
    db += part[((size_t)s * 2 + 1) * H + c];
  }
  if (dweight) dweight[c] = dw;
  if (dbias) dbias[c] = db;
}

constexpr int kMaxSlabs = 128;

}  // namespace

void launch_add_layer_norm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, const uint16_t* bias,
                           float eps, int T, int H, uint16_t* residual_out, uint16_t* out, int sms, cudaStream_t s) {
  const int chunks = (H + kChunk - 1) / kChunk;
  // few rows: one chunk a warp, for the shortest path; many: four, so that an
  // SM holds several rows and their loads overlap
  const int nv = T < 4 * sms && chunks <= 32 ? 1 : 4;
  const dim3 grid((unsigned)T), block(32 * ((chunks + nv - 1) / nv));
  launch_pdl(nv == 1 ? add_layer_norm_kernel<1> : add_layer_norm_kernel<4>, grid, block, 0, s, x, residual, weight,
             bias, eps, H, residual_out, out);
}

size_t norm_backward_scratch_bytes(int T, int H) {
  return sizeof(float2) * (size_t)T + sizeof(float) * 2 * (size_t)H * kMaxSlabs;
}

void launch_norm_backward(const uint16_t* v, const uint16_t* dout, const uint16_t* dresidual, const uint16_t* weight,
                          float eps, int T, int H, bool centre, uint16_t* dx, float* dweight, float* dbias, void* scratch,
                          int sms, cudaStream_t s) {
  const int chunks = (H + kChunk - 1) / kChunk;
  const int nv = T < 4 * sms && chunks <= 32 ? 1 : 4;
  float* part = static_cast<float*>(scratch);
  float2* stats = reinterpret_cast<float2*>(part + 2 * (size_t)H * kMaxSlabs);
  launch_pdl(nv == 1 ? norm_dx_kernel<1> : norm_dx_kernel<4>, dim3((unsigned)T), dim3(32 * ((chunks + nv - 1) / nv)), 0,
             s, v, dout, dresidual, weight, eps, H, (int)centre, dx, stats);
  if (!dweight && !dbias) return;
  const int slab_rows = (T + kMaxSlabs - 1) / kMaxSlabs, slabs = (T + slab_rows - 1) / slab_rows;
  launch_pdl(norm_columns_kernel, dim3((H + 255) / 256, slabs), dim3(128), 0, s, v, dout, (const float2*)stats, T, H,
             slab_rows, part);
  launch_pdl(norm_columns_sum_kernel, dim3((H + 127) / 128), dim3(128), 0, s, (const float*)part, slabs, H, dweight,
             dbias);
}

}  // namespace moe
