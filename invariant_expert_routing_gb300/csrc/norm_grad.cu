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
// Sums over a row have one order for a given H, whatever the batch.  The forward's:
// eight elements in turn, the 32 groups of a 256-element chunk by a fixed tree, the
// chunks by another.
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
                          const uint16_t* __restrict__ bias, float eps, int T, int H, uint16_t* residual_out, uint16_t* out) {
  // (rows shorter than 2048 share a CTA of 256 threads, blockDim.y of them)
  __shared__ float s_sums[kThreads == 256 ? 8 : 1][2][kThreads == 256 ? 32 : kMaxChunks];
  auto s_sum = s_sums[threadIdx.y];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int chunks = (H + kChunk - 1) / kChunk, t = blockIdx.x * blockDim.y + threadIdx.y;
  if (t >= T) H = 0;   // nothing to read or write, but the barriers
  const size_t row = (size_t)t * H;
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
// A warp holds two chunks of a row, and its columns' sums over all rows of the
// CTA, in registers; the rows behind it are on their way into shared memory
// (cp.async: a thread copies what it reads itself, so no barrier is needed for
// them): two rows at a time with two behind them left memory idle
// (192 us for 16448 rows of 7168).  One barrier a row: it carries the row's
// second moments together with the next row's sums, whose values stay in
// registers (one chunk a warp, read twice: 173 us, by instruction issue).  Each
// byte moves once.
constexpr int kFusedMaxChunks = 32, kFusedMaxWarps = 16;
// Rows in shared memory: 192 KB with 512 threads on the SM, in one CTA or in two.  Five,
// which 480 threads leave room for, were no faster (16448 rows of 7168: 153.5 us for
// 154.5, of 5120 and 7680 the same; the RMS norm with dbias 202 for 189).
constexpr int kRing = 4;

// Sums of four values over the CTA, known to every thread: lane halves and
// quarters exchange values, so that each eighth lane group ends with one of the
// four; then 8 lanes a value add the warps' sums.  s_sum: one array a call.
__device__ __forceinline__ void block_sum4(float (&q)[4], int warp, int lane, int warps, float (*s_sum)[kFusedMaxWarps]) {
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
  for (int c = 0; c < kFusedMaxWarps; c += 8)
    if (c + (lane & 7) < warps) t += s_sum[lane >> 3][c + (lane & 7)];
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

// What is summed over the rows: nothing, dout n (16 registers fewer, without which
// the RMS norm's sums would spill: 192 us for 151), and dout.
enum Sums { kNone, kWeight, kBoth };

// part [grid][2][H]: each CTA's sums over its rows (blockIdx.x + i gridDim.x) of
// dout n and dout.  dx may be dresidual (no __restrict__): a row is copied
// before it is written, by the same thread.
template <bool kCentre, Sums kSums, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads)
    norm_backward_kernel(const uint16_t* v_in, const uint16_t* dout, const uint16_t* dresidual,
                         const uint16_t* __restrict__ weight, float eps, int T, int H, uint16_t* dx,
                         float* __restrict__ part) {
  extern __shared__ __align__(16) uint8_t ring[];   // [kRing][3][2][threads] of 16 bytes
  __shared__ float s_sum[2][4][kFusedMaxWarps];     // by the parity of the row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int c[2] = {(int)threadIdx.x * 8, (int)(threadIdx.x + blockDim.x) * 8};   // this thread's columns
  const bool in[2] = {c[0] < H, c[1] < H};
  const int rows = (int)blockIdx.x < T ? (T - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  const uint8_t* own = ring + threadIdx.x * 16;
  const uint32_t mine = smem_u32(own), plane = blockDim.x * 16;
  const size_t stride = (size_t)gridDim.x * H;
  size_t ahead = (size_t)blockIdx.x * H;   // the row to request next
  int asked = 0;
  auto request = [&](uint32_t slot) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool have = in[h] && asked < rows;
      const size_t a = have ? ahead + c[h] : 0;
      const uint32_t dst = mine + (slot * 6 + h) * plane, n = have ? 16 : 0;
      cp_async16(dst, v_in + a, n);
      cp_async16(dst + 2 * plane, dout + a, n);
      if (dresidual) cp_async16(dst + 4 * plane, dresidual + a, n);
    }
    cp_async_commit();
    ahead += stride;
    ++asked;
  };
  auto piece = [&](uint32_t slot, int tensor, int h, F2 (&v)[4]) {
    unpack(*reinterpret_cast<const uint4*>(own + (slot * 6 + tensor * 2 + h) * plane), v);
  };
  pdl_wait();
  pdl_trigger();
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) request(i);
  const float per = 1.0f / (float)H;
  F2 w[2][4], dw[2][4] = {}, db[2][4] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h)
    unpack(in[h] ? __ldg(reinterpret_cast<const uint4*>(weight + c[h])) : make_uint4(0, 0, 0, 0), w[h]);
  // the row in a slot, and the sums of v and g = dout w (unused for the RMS norm)
  auto read = [&](uint32_t slot, F2 (&v)[2][4], F2 (&o)[2][4], float& sv, float& sg) {
    F2 tv = both(0.0f), tg = both(0.0f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      piece(slot, 0, h, v[h]);
      piece(slot, 1, h, o[h]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        tv = add(tv, v[h][j]);
        tg = fma(o[h][j], w[h][j], tg);
        if (kSums == kBoth) db[h][j] = add(db[h][j], o[h][j]);
      }
    }
    sv = total(tv);
    sg = total(tg);
  };
  F2 d[2][4], o[2][4];
  float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  cp_async_wait<kRing - 2>();
  read(0, d, o, q[2], q[3]);
  if (kCentre) block_sum4(q, warp, lane, warps, s_sum[1]);
  float mean = q[2] * per, mean_g = q[3] * per;
  uint32_t slot = 0;
  size_t at = (size_t)blockIdx.x * H;
  for (int i = 0; i < rows; ++i) {
    const uint32_t behind = slot == 0 ? kRing - 1 : slot - 1, next = slot == kRing - 1 ? 0 : slot + 1;
    request(behind);              // into the slot of the row before
    cp_async_wait<kRing - 2>();   // this row and the next
    F2 dd = both(0.0f), dg = both(0.0f);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const F2 minus = both(in[h] ? -mean : 0.0f);   // (past H everything stays zero)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kCentre) d[h][j] = add(d[h][j], minus);
        dd = fma(d[h][j], d[h][j], dd);
        dg = fma(d[h][j], mul(o[h][j], w[h][j]), dg);
      }
    }
    q[0] = total(dd);
    q[1] = total(dg);
    F2 dn[2][4], on[2][4];
    read(next, dn, on, q[2], q[3]);
    block_sum4(q, warp, lane, warps, s_sum[i & 1]);
    const float inv = 1.0f / sqrtf(q[0] * per + eps);
    const float slope = q[1] * per * inv * inv;   // mean(g n) / root
    const F2 inv2 = both(inv), slope2 = both(-slope), minus_g = both(-mean_g);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      F2 r[4] = {};
      if (dresidual) piece(slot, 2, h, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (kSums != kNone) dw[h][j] = fma(o[h][j], mul(d[h][j], inv2), dw[h][j]);
        const F2 g = kCentre ? fma(o[h][j], w[h][j], minus_g) : mul(o[h][j], w[h][j]);
        r[j] = fma(fma(d[h][j], slope2, g), inv2, r[j]);
      }
      if (in[h]) __stcs(reinterpret_cast<uint4*>(dx + at + c[h]), pack(r));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[h][j] = dn[h][j];
        o[h][j] = on[h][j];
      }
    }
    mean = q[2] * per;
    mean_g = q[3] * per;
    slot = next;
    at += stride;
  }
  cp_async_wait<0>();
  if (kSums != kNone) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        if (!in[h]) break;
        float* to = part + (size_t)blockIdx.x * 2 * H + c[h] + 2 * j;
        *reinterpret_cast<ulonglong2*>(to) = make_ulonglong2(dw[h][j].v, dw[h][j + 1].v);
        if (kSums == kBoth) *reinterpret_cast<ulonglong2*>(to + H) = make_ulonglong2(db[h][j].v, db[h][j + 1].v);
      }
  }
}

// ---- rows up to 16384 wide: a CTA an SM, four pieces of eight columns a thread
// whose sums stay in registers, the row in shared memory (read there by the thread
// that copied it) with one or two behind it, and a barrier for each pair of
// moments.  8192 rows of 12288: 171 us, of 16384: 194 (4.7 and
// 5.5 TB/s; dv and slabs of rows, as below: 351 and 411).
constexpr int kWideMaxChunks = 64, kWideThreads = 512;

template <bool kCentre, Sums kSums>
__global__ void __launch_bounds__(kWideThreads, 1)
    norm_backward_wide_kernel(const uint16_t* v_in, const uint16_t* dout, const uint16_t* dresidual,
                              const uint16_t* __restrict__ weight, float eps, int T, int H, int slots, uint16_t* dx,
                              float* __restrict__ part) {
  extern __shared__ __align__(16) uint8_t ring[];   // [slots][3][H] bf16
  __shared__ float s_sum[2][2][4][kFusedMaxWarps];  // by the parity of the row and the moments
  constexpr int kPieces = 4, kStep = 8 * kWideThreads, kWarps = kWideThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = (int)threadIdx.x * 8;
  const int rows = (int)blockIdx.x < T ? (T - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  const size_t stride = (size_t)gridDim.x * H;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  size_t ahead = (size_t)blockIdx.x * H;   // the row to request next
  int asked = 0;
  auto request = [&](int slot) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int c = c0 + k * kStep;
      if (c >= H || asked >= rows) continue;
      const uint32_t dst = smem_u32(ring) + ((uint32_t)slot * 3 * H + c) * 2;
      cp_async16(dst, v_in + ahead + c, 16);
      cp_async16(dst + 2 * H, dout + ahead + c, 16);
      if (dresidual) cp_async16(dst + 4 * H, dresidual + ahead + c, 16);
    }
    cp_async_commit();
    ahead += stride;
    ++asked;
  };
  auto piece = [&](int slot, int tensor, int k, F2 (&v)[4]) {
    const int c = c0 + k * kStep;
    uint4 got = zero;
    if (c < H) got = *reinterpret_cast<const uint4*>(ring + ((size_t)(slot * 3 + tensor) * H + c) * 2);
    unpack(got, v);
  };
  pdl_wait();
  pdl_trigger();
  for (int i = 0; i < slots; ++i) request(i);
  const float per = 1.0f / (float)H;
  uint4 wv[kPieces];
  F2 dw[kPieces][4] = {}, db[kPieces][4] = {};
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    wv[k] = zero;
    if (c0 + k * kStep < H) wv[k] = __ldg(reinterpret_cast<const uint4*>(weight + c0 + k * kStep));
  }
  int slot = 0;
  size_t at = (size_t)blockIdx.x * H;
  for (int i = 0; i < rows; ++i) {
    if (slots == 3)
      cp_async_wait<2>();
    else
      cp_async_wait<1>();
    float mean = 0.0f, mean_g = 0.0f, q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (kCentre) {
      F2 tv = both(0.0f), tg = both(0.0f);
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        F2 v[4], o[4], w[4];
        piece(slot, 0, k, v);
        piece(slot, 1, k, o);
        unpack(wv[k], w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tv = add(tv, v[j]);
          tg = fma(o[j], w[j], tg);
        }
      }
      q[0] = total(tv);
      q[1] = total(tg);
      block_sum4(q, warp, lane, kWarps, s_sum[i & 1][0]);
      mean = q[0] * per;
      mean_g = q[1] * per;
    }
    F2 dd = both(0.0f), dg = both(0.0f);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      F2 v[4], o[4], w[4];
      piece(slot, 0, k, v);
      piece(slot, 1, k, o);
      unpack(wv[k], w);
      const F2 minus = both(c0 + k * kStep < H ? -mean : 0.0f);   // (past H everything stays zero)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 d = kCentre ? add(v[j], minus) : v[j];
        dd = fma(d, d, dd);
        dg = fma(d, mul(o[j], w[j]), dg);
      }
    }
    q[0] = total(dd);
    q[1] = total(dg);
    q[2] = q[3] = 0.0f;
    block_sum4(q, warp, lane, kWarps, s_sum[i & 1][1]);
    const float inv = 1.0f / sqrtf(q[0] * per + eps);
    const float slope = q[1] * per * inv * inv;   // mean(g n) / root
    const F2 inv2 = both(inv), slope2 = both(-slope), minus_g = both(-mean_g), minus = both(-mean);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      if (c0 + k * kStep >= H) continue;
      F2 v[4], o[4], w[4], r[4] = {};
      piece(slot, 0, k, v);
      piece(slot, 1, k, o);
      unpack(wv[k], w);
      if (dresidual) piece(slot, 2, k, r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F2 d = kCentre ? add(v[j], minus) : v[j];
        if (kSums != kNone) dw[k][j] = fma(o[j], mul(d, inv2), dw[k][j]);
        if (kSums == kBoth) db[k][j] = add(db[k][j], o[j]);
        const F2 g = kCentre ? fma(o[j], w[j], minus_g) : mul(o[j], w[j]);
        r[j] = fma(fma(d, slope2, g), inv2, r[j]);
      }
      __stcs(reinterpret_cast<uint4*>(dx + at + c0 + k * kStep), pack(r));
    }
    __syncwarp();
    request(slot);   // into this row's slot, by the threads that have read it
    slot = slot + 1 == slots ? 0 : slot + 1;
    at += stride;
  }
  cp_async_wait<0>();
  if (kSums != kNone) {
#pragma unroll
    for (int k = 0; k < kPieces; ++k)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        if (c0 + k * kStep >= H) break;
        float* to = part + (size_t)blockIdx.x * 2 * H + c0 + k * kStep + 2 * j;
        *reinterpret_cast<ulonglong2*>(to) = make_ulonglong2(dw[k][j].v, dw[k][j + 1].v);
        if (kSums == kBoth) *reinterpret_cast<ulonglong2*>(to + H) = make_ulonglong2(db[k][j].v, db[k][j + 1].v);
      }
  }
}

// ---- wider rows: dv, then the columns' sums in slabs of rows (12 bytes an
// element instead of 8)
// dv of one row a CTA, and the row's (mean, 1 / root) for the weight's gradient.
// dx may be dresidual (no __restrict__): a row is read before the first barrier.
template <int NV, int kThreads>
__global__ void __launch_bounds__(kThreads)
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
    vv[i] = c < H ? __ldcs(reinterpret_cast<const uint4*>(v_in + row + c)) : zero;
    gv[i] = c < H ? __ldcs(reinterpret_cast<const uint4*>(dout + row + c)) : zero;
    rv[i] = c < H && dresidual ? __ldcs(reinterpret_cast<const uint4*>(dresidual + row + c)) : zero;
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

// part[slab][0 / 1][H]: sums over the rows of a slab of dout n and dout; eight
// columns a thread, four rows' loads in flight.
__global__ void __launch_bounds__(128)
    norm_columns_kernel(const uint16_t* __restrict__ v_in, const uint16_t* __restrict__ dout,
                        const float2* __restrict__ stats, int T, int H, int slab_rows, float* __restrict__ part) {
  const int c = (blockIdx.x * 128 + threadIdx.x) * 8;
  pdl_wait();
  pdl_trigger();
  if (c >= H) return;
  const int t0 = blockIdx.y * slab_rows, t1 = min(T, t0 + slab_rows);
  F2 dw[4] = {}, db[4] = {};
  for (int t = t0; t < t1; t += 4) {
    uint4 vv[4], dd[4];
    float2 st[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool have = t + k < t1;
      const size_t at = (size_t)(have ? t + k : t) * H + c;
      vv[k] = __ldcs(reinterpret_cast<const uint4*>(v_in + at));
      dd[k] = have ? __ldcs(reinterpret_cast<const uint4*>(dout + at)) : make_uint4(0, 0, 0, 0);
      st[k] = stats[have ? t + k : t];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (t + k >= t1) break;
      F2 v[4], d[4];
      unpack(vv[k], v);
      unpack(dd[k], d);
      const F2 minus = both(-st[k].x), inv = both(st[k].y);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dw[j] = fma(d[j], mul(add(v[j], minus), inv), dw[j]);
        db[j] = add(db[j], d[j]);
      }
    }
  }
  float* at = part + (size_t)blockIdx.y * 2 * H + c;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    *reinterpret_cast<ulonglong2*>(at + 2 * j) = make_ulonglong2(dw[j].v, dw[j + 1].v);
    *reinterpret_cast<ulonglong2*>(at + H + 2 * j) = make_ulonglong2(db[j].v, db[j + 1].v);
  }
}

// 32 columns a CTA: a warp takes every kWarps-th slab in turn, then those by a tree.
// 16 warps for the 152 slabs of wide rows (all CTAs at once: 2 us less for rows of
// 7168), 32 for more (rows of 1024: 25 us for 30).
template <int kWarps>
__global__ void __launch_bounds__(32 * kWarps)
    norm_columns_sum_kernel(const float* __restrict__ part, int slabs, int H, float* __restrict__ dweight,
                            float* __restrict__ dbias) {
  __shared__ float s[kWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const float* from = part + (size_t)blockIdx.y * H;   // blockIdx.y: 0 dweight, 1 dbias
  float* out = blockIdx.y ? dbias : dweight;
  pdl_wait();
  pdl_trigger();
  if (!out) return;
  float t = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int i = warp; i < slabs; i += kWarps) t += from[(size_t)i * 2 * H + c];
  }
  s[warp][lane] = t;
  __syncthreads();
  constexpr int kSpan = 32 / kWarps;                        // columns a warp joins at once
  const int col = warp * kSpan + lane / kWarps;
  t = s[lane % kWarps][col];
#pragma unroll
  for (int off = kWarps / 2; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
  if (lane % kWarps == 0 && blockIdx.x * 32 + col < H) out[blockIdx.x * 32 + col] = t;
}

constexpr int kMaxSlabs = 128;

}  // namespace

void launch_add_layer_norm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, const uint16_t* bias,
                           float eps, int T, int H, uint16_t* residual_out, uint16_t* out, int sms, cudaStream_t s) {
  const int chunks = (H + kChunk - 1) / kChunk;
  auto go = [&](auto kernel, int nv, int rows) {
    launch_pdl(kernel, dim3((unsigned)((T + rows - 1) / rows)), dim3(32 * ((chunks + nv - 1) / nv), rows), 0, s, x,
               residual, weight, bias, eps, T, H, residual_out, out);
  };
  // few rows: one chunk a warp, for the shortest path; many: four, so that an
  // SM holds several rows and their loads overlap
  if (T < 4 * sms && chunks <= 32)
    go(add_layer_norm_kernel<1, 1024, 1>, 1, 1);
  else if (chunks <= 32)
    go(add_layer_norm_kernel<4, 256, 4>, 4, 8 / ((chunks + 3) / 4));
  else if (chunks <= 64)
    go(add_layer_norm_kernel<4, 512, 2>, 4, 1);
  else
    go(add_layer_norm_kernel<4, 1024, 1>, 4, 1);
}

// The fused kernel's threads for rows of H, and CTAs: as many as fill 152 SMs
// once (a constant, so that the columns' sums have one order for a size).
int fused_threads(int H) { return 32 * ((H + 2 * kChunk - 1) / (2 * kChunk)); }
// Short rows take at least eight a CTA where there are many, so that the sums of
// the CTAs stay few.
int fused_ctas(int H, int T) {
  if ((H + kChunk - 1) / kChunk > kFusedMaxChunks) return T < 152 ? T : 152;   // (the wide kernel)
  const int most = 152 * (512 / fused_threads(H)), eighth = T / 8 > 152 ? T / 8 : 152;
  const int ctas = most < eighth ? most : eighth;
  return T < ctas ? T : ctas;
}

size_t norm_backward_scratch_bytes(int T, int H) {
  if ((H + kChunk - 1) / kChunk <= kWideMaxChunks) return sizeof(float) * 2 * (size_t)H * fused_ctas(H, T);
  return sizeof(float2) * (size_t)T + sizeof(float) * 2 * (size_t)H * kMaxSlabs;
}

template <bool kCentre, Sums kSums>
void launch_wide(const uint16_t* v, const uint16_t* dout, const uint16_t* dresidual, const uint16_t* weight, float eps,
                 int T, int H, uint16_t* dx, float* part, int ctas, cudaStream_t s) {
  auto kernel = norm_backward_wide_kernel<kCentre, kSums>;
  constexpr int kMost = 3 * 6 * 12288;   // bytes of three rows, more than two of 16384
  const int slots = H <= 12288 ? 3 : 2;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  launch_pdl(kernel, dim3(ctas), dim3(kWideThreads), slots * 6 * H, s, v, dout, dresidual, weight, eps, T, H, slots, dx, part);
}

template <bool kCentre, Sums kSums, int kThreads>
void launch_fused(const uint16_t* v, const uint16_t* dout, const uint16_t* dresidual, const uint16_t* weight, float eps,
                  int T, int H, uint16_t* dx, float* part, int ctas, cudaStream_t s) {
  auto kernel = norm_backward_kernel<kCentre, kSums, kThreads>;
  const int threads = fused_threads(H), smem = kRing * 6 * 16 * threads;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing * 6 * 16 * kThreads);
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
  if (chunks <= kWideMaxChunks) {
    slabs = fused_ctas(H, T);
    auto go = [&](auto kernel) { kernel(v, dout, dresidual, weight, eps, T, H, dx, part, slabs, s); };
    auto sized = [&](auto c, auto n) {
      constexpr bool kCentre = decltype(c)::value;
      constexpr Sums kSums = decltype(n)::value;
      if (chunks <= 16)
        go(launch_fused<kCentre, kSums, 256>);
      else if (chunks <= kFusedMaxChunks)
        go(launch_fused<kCentre, kSums, 512>);
      else
        go(launch_wide<kCentre, kSums>);
    };
    using No = std::integral_constant<Sums, kNone>;
    using W = std::integral_constant<Sums, kWeight>;
    using WB = std::integral_constant<Sums, kBoth>;
    if (centre)
      params ? sized(std::true_type{}, WB{}) : sized(std::true_type{}, No{});
    else if (dbias)
      sized(std::false_type{}, WB{});
    else
      dweight ? sized(std::false_type{}, W{}) : sized(std::false_type{}, No{});
  } else {
    float2* stats = reinterpret_cast<float2*>(part + 2 * (size_t)H * kMaxSlabs);
    launch_pdl(norm_dx_kernel<4, 1024>, dim3((unsigned)T), dim3(32 * ((chunks + 3) / 4)), 0, s, v, dout, dresidual, weight,
               eps, H, (int)centre, dx, stats);
    const int slab_rows = (T + kMaxSlabs - 1) / kMaxSlabs;
    slabs = (T + slab_rows - 1) / slab_rows;
    if (params)
      launch_pdl(norm_columns_kernel, dim3((H + 1023) / 1024, slabs), dim3(128), 0, s, v, dout, (const float2*)stats, T, H,
                 slab_rows, part);
  }
  if (params)
    launch_pdl(slabs <= 152 ? norm_columns_sum_kernel<16> : norm_columns_sum_kernel<32>, dim3((H + 31) / 32, 2),
               dim3(slabs <= 152 ? 512 : 1024), 0, s, (const float*)part, slabs, H, dweight, dbias);
}

}  // namespace moe
