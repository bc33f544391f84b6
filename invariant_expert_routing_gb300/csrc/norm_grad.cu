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
#include <type_traits>

#include "bf16x8.cuh"
#include "kernels.h"
#include "pdl.cuh"
#include "ptx.cuh"

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
// kThreads: the most it is launched with.  weight and bias are read when they are
// needed (the SM's rows share them in L1), so that four rows of 7168 fit an SM's
// registers without spilling (they were asked for first: 212 us for 16448 rows).
template <int NV, int kThreads, int kBlocks>
__global__ void __launch_bounds__(kThreads, kBlocks)
    add_layer_norm_kernel(const uint16_t* x, const uint16_t* residual, const uint16_t* __restrict__ weight,
                          const uint16_t* __restrict__ bias, float eps, int H, uint16_t* residual_out, uint16_t* out) {
  __shared__ float s_sum[2][kMaxChunks];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int chunks = (H + kChunk - 1) / kChunk;
  const size_t row = (size_t)blockIdx.x * H;
  pdl_wait();
  pdl_trigger();
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 xv[NV], rv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (warp + i * warps) * kChunk + lane * 8;
    xv[i] = c < H ? __ldcs(reinterpret_cast<const uint4*>(x + row + c)) : zero;
    rv[i] = c < H && residual ? __ldcs(reinterpret_cast<const uint4*>(residual + row + c)) : zero;
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
    if (c >= H) continue;
    float w[8], b[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(weight + c)), w);
    unpack8(bias ? __ldg(reinterpret_cast<const uint4*>(bias + c)) : zero, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * inv, w[j], b[j]);
    *reinterpret_cast<uint4*>(out + row + c) = pack_bf16(v[i]);
  }
}

// ---- the gradients of rows up to 8192 wide
// A warp holds one chunk of two rows at a time, and its columns' sums over all
// rows of the CTA, in registers; the rows behind them are on their way into
// shared memory (cp.async: a thread copies what it reads itself, so no barrier
// is needed for them).  Each byte moves once: bound by memory.
constexpr int kRing = 4;              // rows in shared memory
constexpr int kRowsAtOnce = 2;
constexpr int kFusedMaxChunks = 32;

// Sums of four values over the CTA, known to every thread: lane halves and
// quarters exchange values, so that each eighth lane group ends with one of the
// four; then 8 lanes a value add the chunks' sums.  s_sum: one array a call.
__device__ __forceinline__ void block_sum4(float (&q)[4], int warp, int lane, int chunks, float (*s_sum)[kFusedMaxChunks]) {
  const bool hi = lane & 16;
  float a = hi ? q[2] : q[0], b = hi ? q[3] : q[1];
  a += __shfl_xor_sync(0xffffffffu, hi ? q[0] : q[2], 16);
  b += __shfl_xor_sync(0xffffffffu, hi ? q[1] : q[3], 16);
  const bool up = lane & 8;
  float t = up ? b : a;
  t += __shfl_xor_sync(0xffffffffu, up ? a : b, 8);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  if ((lane & 7) == 0) s_sum[lane >> 3][warp] = t;
  __syncthreads();
  t = 0.0f;
#pragma unroll
  for (int c = 0; c < kFusedMaxChunks; c += 8)
    if (c + (lane & 7) < chunks) t += s_sum[lane >> 3][c + (lane & 7)];
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = __shfl_sync(0xffffffffu, t, 8 * i);
}

// part [grid][2][H]: each CTA's sums over its rows (blockIdx.x + i gridDim.x) of
// dout n and dout.  dx may be dresidual (no __restrict__): a row is copied
// before it is written, by the same thread.
template <bool kCentre, bool kParams, int kThreads>
__global__ void __launch_bounds__(kThreads)
    norm_backward_kernel(const uint16_t* v_in, const uint16_t* dout, const uint16_t* dresidual,
                         const uint16_t* __restrict__ weight, float eps, int T, int H, uint16_t* dx,
                         float* __restrict__ part) {
  extern __shared__ __align__(16) uint8_t ring[];   // [kRing][3][threads] of 16 bytes
  __shared__ float s_sum[2][2][4][kFusedMaxChunks];  // [pair parity][round]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chunks = blockDim.x >> 5;
  const int c = threadIdx.x * 8;
  const bool in = c < H;
  const int rows = (int)blockIdx.x < T ? (T - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  auto slot = [&](int i, int tensor) { return (uint32_t)(((i % kRing) * 3 + tensor) * blockDim.x * 16); };
  auto at = [&](int i) { return ((size_t)blockIdx.x + (size_t)i * gridDim.x) * H + c; };
  auto request = [&](int i) {   // two rows i, i + 1
#pragma unroll
    for (int k = i; k < i + kRowsAtOnce; ++k) {
      const bool have = in && k < rows;
      const size_t a = have ? at(k) : 0;
      cp_async16(mine + slot(k, 0), v_in + a, have ? 16 : 0);
      cp_async16(mine + slot(k, 1), dout + a, have ? 16 : 0);
      if (dresidual) cp_async16(mine + slot(k, 2), dresidual + a, have ? 16 : 0);
    }
    cp_async_commit();
  };
  pdl_wait();
  pdl_trigger();
  request(0);
  const uint4 wv = in ? __ldg(reinterpret_cast<const uint4*>(weight + c)) : make_uint4(0, 0, 0, 0);
  const float per = 1.0f / (float)H;
  float dw[8] = {}, db[8] = {};
  for (int i = 0; i < rows; i += kRowsAtOnce) {
    request(i + kRowsAtOnce);
    cp_async_wait<1>();
    const uint8_t* own = ring + threadIdx.x * 16;
    auto sums = s_sum[(i / kRowsAtOnce) & 1];
    float d[2][8], g[2][8], w[8], q[4];
    unpack8(wv, w);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      unpack8(*reinterpret_cast<const uint4*>(own + slot(i + k, 0)), d[k]);
      unpack8(*reinterpret_cast<const uint4*>(own + slot(i + k, 1)), g[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (kParams) db[j] += g[k][j];
        g[k][j] *= w[j];
      }
    }
    float mean_g[2] = {0.0f, 0.0f};
    if (kCentre) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        q[2 * k] = q[2 * k + 1] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          q[2 * k] += d[k][j];
          q[2 * k + 1] += g[k][j];
        }
      }
      block_sum4(q, warp, lane, chunks, sums[0]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float mean = q[2 * k] * per;
        mean_g[k] = q[2 * k + 1] * per;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[k][j] = in ? d[k][j] - mean : 0.0f;
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      q[2 * k] = q[2 * k + 1] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        q[2 * k] = fmaf(d[k][j], d[k][j], q[2 * k]);
        q[2 * k + 1] = fmaf(d[k][j], g[k][j], q[2 * k + 1]);
      }
    }
    block_sum4(q, warp, lane, chunks, sums[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (i + k >= rows) break;
      const float inv = 1.0f / sqrtf(q[2 * k] * per + eps);
      const float slope = q[2 * k + 1] * per * inv * inv;   // mean(g n) / root
      if (kParams) {
        float o[8];
        unpack8(*reinterpret_cast<const uint4*>(own + slot(i + k, 1)), o);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = fmaf(o[j], d[k][j] * inv, dw[j]);
      }
      float r[8] = {};
      if (dresidual) unpack8(*reinterpret_cast<const uint4*>(own + slot(i + k, 2)), r);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = fmaf(g[k][j] - mean_g[k] - d[k][j] * slope, inv, r[j]);
      if (in) __stcs(reinterpret_cast<uint4*>(dx + at(i + k)), pack_bf16(r));
    }
  }
  cp_async_wait<0>();
  if (kParams && in) {
    float4* p = reinterpret_cast<float4*>(part + (size_t)blockIdx.x * 2 * H + c);
    p[0] = make_float4(dw[0], dw[1], dw[2], dw[3]);
    p[1] = make_float4(dw[4], dw[5], dw[6], dw[7]);
    p = reinterpret_cast<float4*>(part + ((size_t)blockIdx.x * 2 + 1) * H + c);
    p[0] = make_float4(db[0], db[1], db[2], db[3]);
    p[1] = make_float4(db[4], db[5], db[6], db[7]);
  }
}

// ---- wider rows: dv, then the columns' sums in slabs of rows (12 bytes an
// element instead of 8)
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

// 32 columns a CTA: 32 slabs in turn a warp lane column, then those by a tree.
__global__ void __launch_bounds__(1024)
    norm_columns_sum_kernel(const float* __restrict__ part, int slabs, int H, float* __restrict__ dweight,
                            float* __restrict__ dbias) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* from = part + (size_t)blockIdx.y * H;   // blockIdx.y: 0 dweight, 1 dbias
  float* out = blockIdx.y ? dbias : dweight;
  pdl_wait();
  pdl_trigger();
  if (!out) return;
  float t = 0.0f;
  if (c < H)
    for (int i = y; i < slabs; i += 32) t += from[(size_t)i * 2 * H + c];
  s[y][lane] = t;
  __syncthreads();
  t = s[lane][y];   // lane: the slab group, y: the column
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  if (lane == 0 && blockIdx.x * 32 + y < H) out[blockIdx.x * 32 + y] = t;
}

constexpr int kMaxSlabs = 128;

}  // namespace

void launch_add_layer_norm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, const uint16_t* bias,
                           float eps, int T, int H, uint16_t* residual_out, uint16_t* out, int sms, cudaStream_t s) {
  const int chunks = (H + kChunk - 1) / kChunk;
  const dim3 grid((unsigned)T);
  auto go = [&](auto kernel, int nv) {
    launch_pdl(kernel, grid, dim3(32 * ((chunks + nv - 1) / nv)), 0, s, x, residual, weight, bias, eps, H, residual_out,
               out);
  };
  // few rows: one chunk a warp, for the shortest path; many: four, so that an
  // SM holds several rows and their loads overlap
  if (T < 4 * sms && chunks <= 32)
    go(add_layer_norm_kernel<1, 1024, 1>, 1);
  else if (chunks <= 32)
    go(add_layer_norm_kernel<4, 256, 4>, 4);
  else
    go(add_layer_norm_kernel<4, 1024, 1>, 4);
}

// CTAs of the fused kernel for rows of H: as many as fill 152 SMs once (a
// constant, so that the columns' sums have one order for a size).
int fused_ctas(int H, int T) {
  const int threads = 32 * ((H + kChunk - 1) / kChunk), most = 152 * (1024 / threads);
  return T < most ? T : most;
}

size_t norm_backward_scratch_bytes(int T, int H) {
  if ((H + kChunk - 1) / kChunk <= kFusedMaxChunks) return sizeof(float) * 2 * (size_t)H * fused_ctas(H, T);
  return sizeof(float2) * (size_t)T + sizeof(float) * 2 * (size_t)H * kMaxSlabs;
}

template <bool kCentre, bool kParams, int kThreads>
void launch_fused(const uint16_t* v, const uint16_t* dout, const uint16_t* dresidual, const uint16_t* weight, float eps,
                  int T, int H, uint16_t* dx, float* part, int ctas, cudaStream_t s) {
  auto kernel = norm_backward_kernel<kCentre, kParams, kThreads>;
  const int threads = 32 * ((H + kChunk - 1) / kChunk), smem = kRing * 3 * 16 * threads;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing * 3 * 16 * kThreads);
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  launch_pdl(kernel, dim3(ctas), dim3(threads), smem, s, v, dout, dresidual, weight, eps, T, H, dx, part);
}

void launch_norm_backward(const uint16_t* v, const uint16_t* dout, const uint16_t* dresidual, const uint16_t* weight,
                          float eps, int T, int H, bool centre, uint16_t* dx, float* dweight, float* dbias, void* scratch,
                          cudaStream_t s) {
  const int chunks = (H + kChunk - 1) / kChunk;
  const bool params = dweight || dbias;
  float* part = static_cast<float*>(scratch);
  int slabs;
  if (chunks <= kFusedMaxChunks) {
    slabs = fused_ctas(H, T);
    auto go = [&](auto kernel) { kernel(v, dout, dresidual, weight, eps, T, H, dx, part, slabs, s); };
    // (compiled for the threads it needs: more registers a thread for fewer)
    auto sized = [&](auto c, auto p) {
      if (chunks <= 16)
        go(launch_fused<decltype(c)::value, decltype(p)::value, 512>);
      else if (chunks <= 28)
        go(launch_fused<decltype(c)::value, decltype(p)::value, 896>);
      else
        go(launch_fused<decltype(c)::value, decltype(p)::value, 1024>);
    };
    if (centre)
      params ? sized(std::true_type{}, std::true_type{}) : sized(std::true_type{}, std::false_type{});
    else
      params ? sized(std::false_type{}, std::true_type{}) : sized(std::false_type{}, std::false_type{});
  } else {
    float2* stats = reinterpret_cast<float2*>(part + 2 * (size_t)H * kMaxSlabs);
    launch_pdl(norm_dx_kernel<4>, dim3((unsigned)T), dim3(32 * ((chunks + 3) / 4)), 0, s, v, dout, dresidual, weight, eps,
               H, (int)centre, dx, stats);
    const int slab_rows = (T + kMaxSlabs - 1) / kMaxSlabs;
    slabs = (T + slab_rows - 1) / slab_rows;
    if (params)
      launch_pdl(norm_columns_kernel, dim3((H + 255) / 256, slabs), dim3(128), 0, s, v, dout, (const float2*)stats, T, H,
                 slab_rows, part);
  }
  if (params)
    launch_pdl(norm_columns_sum_kernel, dim3((H + 31) / 32, 2), dim3(1024), 0, s, (const float*)part, slabs, H, dweight,
               dbias);
}

}  // namespace moe
