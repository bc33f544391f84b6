// Grouped SwiGLU expert GEMMs on microscaled 4-bit operands (mx.cuh), on the
// block-scaled tcgen05 tensor path (kind::mxf4, e2m1 x e2m1, E8M0 scales per
// 32 elements of K):
//   W13: [g | u] = X . W13_e,  a = silu(g) * u  ->  codes and scales of a
//   W2 : y = a . W2_e          ->  bf16
// Token rows are operand A (M = 128 TMEM lanes), weight rows operand B (N
// columns), so that a thread of the epilogue holds one token's neighbouring
// features: a block of 32 is quantised in its registers.  Both operands are
// K-major as stored (256 elements a 128-byte swizzled row).  W13 columns
// alternate 32 gate and the same 32 up features.
//
// Every tile runs the same instruction sequence: K from 0 to the end, 64
// elements per MMA, fp32 accumulation in TMEM, no split-K, no atomics; rows
// and columns of an MMA are independent sums, so a token's row does not
// depend on the batch or on the column width of the work item.
//
// Persistent kernel, one CTA per SM, 10 warps:
//   warp 0      TMA producer: codes (tensor maps) and scales (512-byte chunks)
//   warp 1      TMEM allocation; one thread copies the stage's scales into
//               TMEM (tcgen05.cp) and issues the MMAs
//   warps 2..9  epilogue (two warps per TMEM lane quarter)
// Each stage has TMEM columns of its own for its scales: they are rewritten
// only after the commit of the MMAs that read them released the stage.
#include <cuda_bf16.h>
#include <cstdint>

#include "kernels.h"
#include "mx.cuh"
#include "mx_gemm.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace mx;

constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kStageK = 256;                         // elements of K per stage: one 128-byte row
constexpr int kSmallRows = 32;                       // token box of a tile with at most 32 routed rows
constexpr uint32_t kSmemBudget = 226 * 1024;

template <int BN>
struct Cfg {
  static constexpr int kSfbTiles = (BN + kSfRows - 1) / kSfRows;      // 128-row scale tiles of B
  static constexpr uint32_t kABytes = kMxTileRows * 128;
  static constexpr uint32_t kBBytes = BN * 128;
  static constexpr uint32_t kSfaBytes = 2 * kSfChunkBytes;
  static constexpr uint32_t kSfbBytes = kSfbTiles * 2 * kSfChunkBytes;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  static constexpr uint32_t kBarBytes = 512;
  static constexpr int kFit = (int)((kSmemBudget - kBarBytes - 1024) / kStageBytes);
  static constexpr int kStages = kFit < 8 ? kFit : 8;
  static constexpr int kNumAcc = BN <= 128 ? 2 : 1;
  static constexpr uint32_t kSfCols = 8 + 8 * kSfbTiles;               // TMEM columns of a stage's scales
  static constexpr uint32_t kSfCol0 = kNumAcc * BN;
  static constexpr uint32_t kColsUsed = kSfCol0 + kStages * kSfCols;
  static constexpr uint32_t kTmemCols = kColsUsed <= 256 ? 256 : 512;
  static constexpr uint32_t kSmemBytes = kStages * kStageBytes + kBarBytes + 1024;
  static_assert(kColsUsed <= 512, "accumulators and scales fit in TMEM");
  static_assert(kStageBytes % 1024 == 0, "stages stay aligned to the swizzle atom");
};

struct Item {
  int f, tile, expert, row0, valid;
};

// Work item -> (feature tile, token tile): items of one expert are
// contiguous; inside an expert they run in groups of feature tiles x all of
// the expert's token tiles, a group sized so that one wave of CTAs shares its
// weight and token tiles through L2.
__device__ __forceinline__ Item item_of(const MxGemmArgs& a, int item, int num_tiles, int nf) {
  int first = 0, count = num_tiles;
  if (!a.identity_T) {
    const GemmTile g = a.tiles[item / nf];
    first = g.first;
    count = g.count;
  }
  const int l = item - first * nf;
  const int G = max(1, min(nf, (a.concurrent + count - 1) / count));
  const int grp = l / (count * G);
  const int gsz = min(G, nf - grp * G);
  const int lin = l - grp * count * G;
  Item w;
  w.f = grp * G + lin % gsz;
  w.tile = first + lin / gsz;
  if (a.identity_T) {
    w.expert = 0;
    w.row0 = w.tile * kMxTileRows;
    w.valid = min(kMxTileRows, a.identity_T - w.row0);
  } else {
    const GemmTile g = a.tiles[w.tile];
    w.expert = g.expert;
    w.row0 = g.row0;
    w.valid = g.valid;
  }
  return w;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2,
                                            uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3,
                                            int c4, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar), "l"(policy)
      : "memory");
}

// a = silu(g) * u of 32 neighbouring features of one token, quantised:
// 16 bytes of codes, one scale byte.
__device__ __forceinline__ void store_swiglu_block(const float (&g)[32], float (&u)[32], uint8_t* codes,
                                                   uint8_t* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    u[i] = __fdividef(g[i], 1.0f + __expf(-g[i])) * u[i];
    m = max(m, __float_as_uint(u[i]) & 0x7FFFFFFFu);   // orders infinities and NaN above the finite values
  }
  const uint32_t byte = scale_byte(m);
  uint4 c = make_uint4(0, 0, 0, 0);
  if (byte != 255u) {
    const float inv = scale_inverse(byte);
    uint32_t q[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = u[8 * w + i] * inv;
      q[w] = pack8(t);
    }
    c = make_uint4(q[0], q[1], q[2], q[3]);
  }
  *reinterpret_cast<uint4*>(codes) = c;
  *scale = (uint8_t)byte;
}

__device__ __forceinline__ void store_bf16_block(const float (&v)[32], uint16_t* out) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[8 * q + 2 * i], v[8 * q + 2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    reinterpret_cast<uint4*>(out)[q] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <bool kW13, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
                   const __grid_constant__ CUtensorMap x_map_small, const MxGemmArgs args) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t full0 = smem_u32(smem + C::kStages * C::kStageBytes);
  const uint32_t empty0 = full0 + 8 * C::kStages;
  const uint32_t tfull0 = empty0 + 8 * C::kStages;
  const uint32_t tempty0 = tfull0 + 16;
  const uint32_t drain = tempty0 + 16;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kchunks = args.K / kSfChunkK;
  const int ksteps = (args.K + kStageK - 1) / kStageK;
  const int nf = (args.features + BN - 1) / BN;
  const uint64_t wlim = args.wait_ns ? args.wait_ns : kWaitLimitNs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < C::kNumAcc; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, kEpiWarps);
    }
    mbar_init(drain, 1);
    s_abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s_tmem_base), C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&w_map);
    prefetch_tmap(&x_map);
    prefetch_tmap(&x_map_small);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem_base;
  pdl_wait();
  pdl_trigger();
  const int num_tiles =
      args.identity_T ? (args.identity_T + kMxTileRows - 1) / kMxTileRows : *args.num_tiles;
  const int total = num_tiles * nf;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t pol_w = policy_evict_normal();
      const uint64_t pol_x = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      int armed = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
        const Item w = item_of(args, item, num_tiles, nf);
        const bool small = w.valid <= kSmallRows;
        const uint32_t a_tx = (small ? kSmallRows : kMxTileRows) * 128u;
        // scale tiles of B that exist (the last item of an odd number of 128-row tiles has one)
        const int sft0 = w.f * BN / kSfRows;
        const int sft = min(C::kSfbTiles, args.features / kSfRows - sft0);
        const uint8_t* sfa = args.a_sf + (size_t)w.tile * kchunks * kSfChunkBytes;
        const uint8_t* sfb =
            args.b_sf + ((size_t)w.expert * (args.features / kSfRows) + sft0) * kchunks * kSfChunkBytes;
        for (int ks = 0; ks < ksteps; ++ks) {
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1u, &s_abort, wlim)) {
            ok = false;
            break;
          }
          const uint32_t sA = smem_u32(smem + stage * C::kStageBytes);
          const uint32_t sB = sA + C::kABytes;
          const uint32_t sFa = sB + C::kBBytes, sFb = sFa + C::kSfaBytes;
          const uint32_t fb = full0 + 8 * stage;
          const uint32_t sf_bytes = (uint32_t)min(2, kchunks - 2 * ks) * kSfChunkBytes;
          mbar_arrive_expect_tx(fb, a_tx + C::kBBytes + sf_bytes * (1 + sft));
          if (kW13)
            tma_load_5d(sB, &w_map, ks * 128, 0, 0, w.f * (BN / 64), w.expert, fb, pol_w);
          else
            tma_load_3d(sB, &w_map, ks * 128, w.f * BN, w.expert, fb, pol_w);
          tma_load_2d(sA, small ? &x_map_small : &x_map, ks * 128, w.row0, fb, pol_x);
          bulk_load(sFa, sfa + (size_t)(2 * ks) * kSfChunkBytes, sf_bytes, fb);
          for (int t = 0; t < sft; ++t)
            bulk_load(sFb + t * 2 * kSfChunkBytes, sfb + ((size_t)t * kchunks + 2 * ks) * kSfChunkBytes, sf_bytes, fb);
          armed = min(armed + 1, C::kStages);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        s_abort = 1;
        atomicOr(args.status, kDevErrTimeout);
      }
      if (s_abort) {
        // let the copies already issued land before exit
        volatile int no_abort = 0;
        int s = stage;
        uint32_t ph = phase;
        for (int i = 0; i < armed; ++i) {
          if (--s < 0) {
            s = C::kStages - 1;
            ph ^= 1u;
          }
          mbar_wait(full0 + 8 * s, ph, &no_abort);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
        if (!mbar_wait(tempty0 + 8 * acc, acc_phase ^ 1u, &s_abort, wlim)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // an item narrower than a scale tile takes its columns of it
        const int f = (BN < kSfRows) ? item_of(args, item, num_tiles, nf).f : 0;
        const uint32_t sfb_skip = (BN < kSfRows) ? (uint32_t)(f * BN % kSfRows) / 32u : 0u;
        const uint32_t d0 = tmem + acc * BN;
        for (int ks = 0; ks < ksteps; ++ks) {
          if (!mbar_wait(full0 + 8 * stage, phase, &s_abort, wlim)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sA = smem_u32(smem + stage * C::kStageBytes);
          const uint32_t sB = sA + C::kABytes;
          const uint32_t sFa = sB + C::kBBytes, sFb = sFa + C::kSfaBytes;
          const uint32_t ta = tmem + C::kSfCol0 + stage * C::kSfCols, tb = ta + 8;
          const int chunks = min(2, kchunks - 2 * ks);
          // scales: chunk c of A in columns ta + 4c, of B's tile t in tb + (c kSfbTiles + t) 4
          for (int c = 0; c < chunks; ++c) {
            cp_scales(ta + 4 * c, sdesc_scales(sFa + c * kSfChunkBytes));
#pragma unroll
            for (int t = 0; t < C::kSfbTiles; ++t)
              cp_scales(tb + 4 * (c * C::kSfbTiles + t), sdesc_scales(sFb + (2 * t + c) * kSfChunkBytes));
          }
          const uint64_t ad = sdesc_sw128(sA, 16, 1024), bd = sdesc_sw128(sB, 16, 1024);
          for (int c = 0; c < chunks; ++c) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
              mma_mxf4(d0, ad + (2 * c + half) * 2, bd + (2 * c + half) * 2, idesc_mxf4(kMxTileRows, BN, half),
                       ta + 4 * c, tb + 4 * c * C::kSfbTiles + sfb_skip, (ks | c | half) != 0 ? 1u : 0u);
          }
          mma_commit(empty0 + 8 * stage);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(tfull0 + 8 * acc);
        if (++acc == C::kNumAcc) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok) {
        s_abort = 1;
        atomicOr(args.status, kDevErrTimeout);
      }
      // all issued MMAs must be complete before TMEM is released
      mma_commit(drain);
      volatile int no_abort = 0;
      mbar_wait(drain, 0, &no_abort);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;              // TMEM lanes this warp may access
    const int half = (warp - 2) / 4;           // which blocks of columns
    const int r = quarter * 32 + lane;         // token row of the tile
    constexpr int kBlockCols = kW13 ? 64 : 32; // columns of one block (W13: 32 gate, 32 up)
    constexpr int kBlocks = BN / kBlockCols;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
      const Item w = item_of(args, item, num_tiles, nf);
      int got = 1;
      if (lane == 0) got = mbar_wait(tfull0 + 8 * acc, acc_phase, &s_abort, wlim) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) {
        if (lane == 0) {
          s_abort = 1;
          atomicOr(args.status, kDevErrTimeout);
        }
        break;
      }
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(quarter * 32) << 16) + acc * BN;
      const size_t row = (size_t)w.row0 + r;
      if (quarter * 32 < w.valid) {
        for (int b = half; b < kBlocks; b += 2) {
          if (kW13) {
            const int feat = w.f * (BN / 2) + b * 32;
            float g[32], u[32];
            tmem_load32x2(tbase + b * 64, g, tbase + b * 64 + 32, u);
            if (r < w.valid)
              store_swiglu_block(g, u, args.out_codes + (row * args.out_ld + feat) / 2,
                                 args.out_sf + ((size_t)w.tile * (args.out_ld / kSfChunkK) + feat / kSfChunkK) * kSfChunkBytes +
                                     sf_row_offset(r) + (feat % kSfChunkK) / kBlock);
          } else {
            const int feat = w.f * BN + b * 32;
            if (feat >= args.features) break;
            float v[32];
            tmem_load32(tbase + b * 32, v);
            if (r < w.valid) store_bf16_block(v, args.out + row * args.out_ld + feat);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tempty0 + 8 * acc);
      if (++acc == C::kNumAcc) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

template <bool kW13, int BN>
void launch(const CUtensorMap& w_map, const CUtensorMap& x_map, const CUtensorMap& x_small, MxGemmArgs a,
            int64_t max_tiles, int sms, cudaStream_t s) {
  auto kernel = mx_gemm_kernel<kW13, BN>;
  constexpr int smem = (int)Cfg<BN>::kSmemBytes;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int64_t items = max_tiles * ((a.features + BN - 1) / BN);
  if (items <= 0) return;
  const int grid = (int)(items < sms ? items : sms);
  a.concurrent = grid;
  launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, s, w_map, x_map, x_small, a);
}

// Routed rows in tile order: a warp a row (16 bytes of codes a lane, then one
// 4-byte word of scales per 128 elements, placed by sf_row_offset).
constexpr int kGatherWarps = 8;
__global__ void __launch_bounds__(32 * kGatherWarps) mx_gather_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, const int32_t* __restrict__ sorted, int slots,
    int T, int H, const GemmTile* __restrict__ tiles, const int32_t* __restrict__ num_tiles, int identity_T,
    uint8_t* __restrict__ x_perm, uint8_t* __restrict__ x_sf) {
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = identity_T ? (identity_T + kMxTileRows - 1) / kMxTileRows : *num_tiles;
  const int kchunks = H / kSfChunkK;
  const long long R = (long long)T * slots;
  const long long rows = (long long)n * kMxTileRows;
  const long long step = (long long)gridDim.x * kGatherWarps;
  for (long long i = (long long)blockIdx.x * kGatherWarps + warp; i < rows; i += step) {
    const int tile = (int)(i / kMxTileRows), r = (int)(i % kMxTileRows);
    long long token;
    size_t row = (size_t)i;
    if (identity_T) {
      if (i >= identity_T) continue;
      token = i;
    } else {
      if (r >= tiles[tile].valid) continue;
      row = (size_t)tiles[tile].row0 + r;
      const int id = sorted[row];
      if (id < 0 || id >= R) continue;
      token = id / slots;
      const uint4* src = reinterpret_cast<const uint4*>(codes + token * (H / 2));
      uint4* dst = reinterpret_cast<uint4*>(x_perm + row * (H / 2));
      for (int c = lane; c < H / 32; c += 32) dst[c] = __ldg(src + c);
    }
    const uint32_t* ssrc = reinterpret_cast<const uint32_t*>(scales + token * (H / kBlock));
    for (int c = lane; c < kchunks; c += 32)
      *reinterpret_cast<uint32_t*>(x_sf + ((size_t)tile * kchunks + c) * kSfChunkBytes + sf_row_offset(r)) = __ldg(ssrc + c);
  }
}

}  // namespace

bool mx_gemm_smem_ok() {
  int dev = 0, optin = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  return optin >= (int)Cfg<256>::kSmemBytes && optin >= (int)Cfg<64>::kSmemBytes;
}

int mx_tile_features(bool w13, int features, int64_t max_tiles, int sms) {
  (void)w13;
  const int64_t wide = max_tiles * ((features + 255) / 256);
  return wide >= 2 * sms ? 256 : 64;
}

void launch_mx_gemm(bool w13, const CUtensorMap& w_map, const CUtensorMap& x_map, const CUtensorMap& x_small,
                    const MxGemmArgs& a, int64_t max_tiles, int sms, cudaStream_t s) {
  if (a.tile_features == 256) {
    if (w13)
      launch<true, 256>(w_map, x_map, x_small, a, max_tiles, sms, s);
    else
      launch<false, 256>(w_map, x_map, x_small, a, max_tiles, sms, s);
  } else {
    if (w13)
      launch<true, 64>(w_map, x_map, x_small, a, max_tiles, sms, s);
    else
      launch<false, 64>(w_map, x_map, x_small, a, max_tiles, sms, s);
  }
}

void launch_mx_gather(const uint8_t* codes, const uint8_t* scales, const int32_t* sorted_route_ids, int slots,
                      int T, int H, const GemmTile* tiles, const int32_t* num_tiles, int identity_T,
                      int64_t max_tiles, uint8_t* x_perm, uint8_t* x_sf, cudaStream_t s) {
  const int64_t blocks = max_tiles * kMxTileRows / kGatherWarps;
  const int grid = (int)(blocks < 152 * 8 ? blocks : 152 * 8);
  launch_pdl(mx_gather_kernel, dim3(grid), dim3(32 * kGatherWarps), 0, s, codes, scales, sorted_route_ids, slots, T, H,
             tiles, num_tiles, identity_T, x_perm, x_sf);
}

}  // namespace moe
