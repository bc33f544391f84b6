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
// A warp holds one chunk of a row, and its columns' sums over all rows of the
// CTA, in registers; the rows behind it are on their way into shared memory
// (cp.async: a thread copies what it reads itself, so no barrier is needed for
// them), as many as fit: two rows at a time with two behind them left memory idle
// (192 us for 16448 rows of 7168).  One barrier a row: it carries the row's
// second moments together with the next row's sums.  Each byte moves once: bound
// by memory.
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

// Two fp32 values in one 64-bit register: an add, product or fma of both is one
// instruction (the kernel issues two thirds of what it would one by one).
struct F2 {
  unsigned long long v = 0;
};
__device__ __forceinline__ F2 pair(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 both(float x) { return pair(x, x); }
__device__ __forceinline__ float2 parts(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ float total(F2 a) {
  const float2 p = parts(a);
  return p.x + p.y;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ void unpack(const uint4& p, F2 (&v)[4]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack(const F2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = parts(v[i]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// part [grid][2][H]: each CTA's sums over its rows (blockIdx.x + i gridDim.x) of
// dout n and dout.  dx may be dresidual (no __restrict__): a row is copied
// before it is written, by the same thread.
template <bool kCentre, bool kParams, int kThreads, int kRing>
__global__ void __launch_bounds__(kThreads)
    norm_backward_kernel(const uint16_t* v_in, const uint16_t* dout, const uint16_t* dresidual,
                         const uint16_t* __restrict__ weight, float eps, int T, int H, uint16_t* dx,
                         float* __restrict__ part) {
  extern __shared__ __align__(16) uint8_t ring[];   // [kRing][3][threads] of 16 bytes
  __shared__ float s_sum[2][4][kFusedMaxChunks];    // by the parity of the row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, chunks = blockDim.x >> 5;
  const int c = threadIdx.x * 8;
  const bool in = c < H;
  const int rows = (int)blockIdx.x < T ? (T - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  const uint8_t* own = ring + threadIdx.x * 16;
  const uint32_t mine = smem_u32(own), plane = blockDim.x * 16;
  auto at = [&](int i) { return ((size_t)blockIdx.x + (size_t)i * gridDim.x) * H + c; };
  auto request = [&](int i, uint32_t slot) {
    const bool have = in && i < rows;
    const size_t a = have ? at(i) : 0;
    const uint32_t dst = mine + slot * 3 * plane, n = have ? 16 : 0;
    cp_async16(dst, v_in + a, n);
    cp_async16(dst + plane, dout + a, n);
    if (dresidual) cp_async16(dst + 2 * plane, dresidual + a, n);
    cp_async_commit();
  };
  auto piece = [&](uint32_t slot, int tensor, F2 (&v)[4]) {
    unpack(*reinterpret_cast<const uint4*>(own + (slot * 3 + tensor) * plane), v);
  };
  pdl_wait();
  pdl_trigger();
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) request(i, i);
  const uint4 wv = in ? __ldg(reinterpret_cast<const uint4*>(weight + c)) : make_uint4(0, 0, 0, 0);
  const float per = 1.0f / (float)H;
  F2 dw[4] = {}, db[4] = {};
  // the sums of v and g of the row in a slot
  auto row_sums = [&](uint32_t slot, float& sv, float& sg) {
    F2 v[4], g[4], w[4];
    piece(slot, 0, v);
    piece(slot, 1, g);
    unpack(wv, w);
    sv = total(add(add(v[0], v[1]), add(v[2], v[3])));
    F2 t = mul(g[0], w[0]);
#pragma unroll
    for (int j = 1; j < 4; ++j) t = fma(g[j], w[j], t);
    sg = total(t);
  };
  float mean = 0.0f, mean_g = 0.0f;
  if (kCentre) {
    cp_async_wait<kRing - 2>();
    float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    row_sums(0, q[2], q[3]);
    block_sum4(q, warp, lane, chunks, s_sum[1]);
    mean = q[2] * per;
    mean_g = q[3] * per;
  }
  uint32_t slot = 0;
  for (int i = 0; i < rows; ++i) {
    const uint32_t behind = slot == 0 ? kRing - 1 : slot - 1, next = slot == kRing - 1 ? 0 : slot + 1;
    request(i + kRing - 1, behind);   // into the slot of the row before
    cp_async_wait<kRing - 2>();       // this row and the next
    F2 d[4], g[4], w[4];
    piece(slot, 0, d);
    piece(slot, 1, g);
    unpack(wv, w);
    const F2 minus = both(in ? -mean : 0.0f);   // (past H everything stays zero)
    F2 dd = both(0.0f), dg = both(0.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kParams) db[j] = add(db[j], g[j]);
      g[j] = mul(g[j], w[j]);
      if (kCentre) d[j] = add(d[j], minus);
      dd = fma(d[j], d[j], dd);
      dg = fma(d[j], g[j], dg);
    }
    float q[4] = {total(dd), total(dg), 0.0f, 0.0f};
    if (kCentre) row_sums(next, q[2], q[3]);
    block_sum4(q, warp, lane, chunks, s_sum[i & 1]);
    const float inv = 1.0f / sqrtf(q[0] * per + eps);
    const float slope = q[1] * per * inv * inv;   // mean(g n) / root
    const F2 inv2 = both(inv), slope2 = both(-slope), minus_g = both(-mean_g);
    if (kParams) {
      F2 o[4];
      piece(slot, 1, o);
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[j] = fma(o[j], mul(d[j], inv2), dw[j]);
    }
    F2 r[4] = {};
    if (dresidual) piece(slot, 2, r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kCentre) g[j] = add(g[j], minus_g);
      r[j] = fma(fma(d[j], slope2, g[j]), inv2, r[j]);
    }
    if (in) __stcs(reinterpret_cast<uint4*>(dx + at(i)), pack(r));
    mean = q[2] * per;
    mean_g = q[3] * per;
    slot = next;
  }
  cp_async_wait<0>();
  if (kParams && in) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      *reinterpret_cast<F2*>(part + (size_t)blockIdx.x * 2 * H + c + 2 * j) = dw[j];
      *reinterpret_cast<F2*>(part + ((size_t)blockIdx.x * 2 + 1) * H + c + 2 * j) = db[j];
    }
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

template <bool kCentre, bool kParams, int kThreads, int kRing>
void launch_fused(const uint16_t* v, const uint16_t* dout, const uint16_t* dresidual, const uint16_t* weight, float eps,
                  int T, int H, uint16_t* dx, float* part, int ctas, cudaStream_t s) {
  auto kernel = norm_backward_kernel<kCentre, kParams, kThreads, kRing>;
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
    // rows in shared memory: what 227 KB hold, of the CTAs on an SM together
    auto sized = [&](auto c, auto p) {
      if (chunks <= 16)
        go(launch_fused<decltype(c)::value, decltype(p)::value, 512, 4>);
      else if (chunks <= 28)
        go(launch_fused<decltype(c)::value, decltype(p)::value, 896, 5>);
      else
        go(launch_fused<decltype(c)::value, decltype(p)::value, 1024, 4>);
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
