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
// Persistent kernels, one CTA per SM:
//   warp 0      TMA producer: codes (tensor maps) and scales (512-byte chunks)
//   warp 1      TMEM allocation; copies the stage's scales into TMEM
//               (tcgen05.cp) and issues the MMAs
//   warp 2      scheduler: looks the work items up ahead of the others
//   warps 4..   epilogue: eight warps, two per TMEM lane quarter (twelve in CTA
//               pairs, three per quarter)
// Every wait is bounded; a CTA in which one ran out ends as pipeline_end.h says.
// Each stage has TMEM columns of its own for its scales (CTA pairs: see
// there): they are rewritten only after the commit of the MMAs that read them
// released the stage.
//
// Three forms, by the average number of rows an expert has (the thresholds
// stand at kSwapMaxRows and kPairMinRows), since what bounds them differs:
//   few rows    operands swapped, 32-row tiles: bound by the weights' bytes.
//               One token on 2 of 8 experts, H 4096, I 14336: a pass 42 us, 187
//               MB; of it W13 19 us (21, 6.3 TB/s, without the front's
//               prefetch), W2 15 us (4.4 TB/s: 64 items; items of 64 rows on
//               128 SMs were 2 us slower).
//   some rows   128-row tiles on single CTAs: weights' bytes again.  512
//               tokens x 8 of 128 experts, H 2048, I 768: a pass 67 us, 337 MB.
//   many rows   CTA pairs, 256-row tiles.  4096 tokens x 2 of 8 experts, H 4096,
//               I 14336: W13 300 us (6.4 PFLOP/s), W2 170 us (5.7); 8192 x 8 of
//               128, H 2048, I 768: W13 84 us, W2 72 us, the latter bound by its
//               400 MB (5.5 TB/s).
#include <cuda_bf16.h>
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "mx.cuh"
#include "mx_gemm.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace mx;

constexpr int kEpiWarps = 8;
constexpr int kRoleWarps = 4;                        // producer, MMA issuer, scheduler, none: the epilogue starts at a lane quarter of 0
constexpr int kThreads = (kRoleWarps + kEpiWarps) * 32;
constexpr int kStageK = 256;                         // elements of K per stage: one 128-byte row
constexpr int kSmallRows = 32;                       // token box of a tile with at most 32 routed rows, rows of a swapped tile
constexpr uint32_t kSmemLimit = 226 * 1024;
// Operands swapped where experts average at most so many rows (H 4096, I
// 14336, 8 experts: swapped 126 us against 132 with 16 rows, 142 against 132
// with 25), CTA pairs from so many on (H 2048, I 768, 128 experts: single CTAs
// 75 us against 83 with 64 rows, 88 against 88 with 96, 97 against 93 with 128).
constexpr int kSwapMaxRows = 16;
constexpr int kPairMinRows = 96;
// Wide work items (256 weight rows, else 128, else 64) while they come to so
// many per SM: 512 tokens x 8 of 128 experts, 5 waves of wide W13 items 69.3 us
// a pass, 10 of 128 rows 67.4 us.
constexpr int kMinWaves = 8;
constexpr uint32_t kSfUnits = kSfChunkBytes >> 4;    // a scale chunk in descriptor units

// BN weight rows a work item.  kSwap (tiles of at most 32 token rows): the
// weight rows are operand A and the tokens operand B (see below).
template <int BN, bool kSwap>
struct Cfg {
  static_assert(!kSwap || BN == 128, "swapped items have the 128 rows of an MMA");
  static constexpr int kTokens = kSwap ? kSmallRows : kMxTileRows;    // token rows of a tile
  static constexpr int kSfbTiles = (BN + kSfRows - 1) / kSfRows;      // 128-row scale tiles of the weights
  static constexpr uint32_t kABytes = kTokens * 128;
  static constexpr uint32_t kBBytes = BN * 128;
  static constexpr uint32_t kSfaBytes = 2 * kSfChunkBytes;
  static constexpr uint32_t kSfbBytes = kSfbTiles * 2 * kSfChunkBytes;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  static constexpr uint32_t kXchgBytes = kSwap ? 2 * 2 * 16 * 32 * 4 : 0;   // up values handed to the gate warps
  static constexpr uint32_t kBarBytes = 512;
  static constexpr int kFit = (int)((kSmemLimit - kBarBytes - kXchgBytes - 1024) / kStageBytes);
  static constexpr int kMaxStages = kSwap ? 9 : 8;
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static constexpr int kCols = kSwap ? kTokens : BN;                   // columns of an accumulator
  static constexpr int kNumAcc = kCols <= 128 ? 2 : 1;
  static constexpr uint32_t kSfCols = 8 + 8 * kSfbTiles;               // TMEM columns of a stage's scales
  static constexpr uint32_t kSfCol0 = kNumAcc * kCols;
  static constexpr uint32_t kColsUsed = kSfCol0 + kStages * kSfCols;
  static constexpr uint32_t kTmemCols = kColsUsed <= 256 ? 256 : 512;
  static constexpr uint32_t kSmemBytes = kStages * kStageBytes + kXchgBytes + kBarBytes + 1024;
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
template <int kRows = kMxTileRows>
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
    w.row0 = w.tile * kRows;
    w.valid = min(kRows, a.identity_T - w.row0);
  } else {
    const GemmTile g = a.tiles[w.tile];
    w.expert = g.expert;
    w.row0 = g.row0;
    w.valid = g.valid;
  }
  return w;
}

// Items reach the warps of a CTA through a ring in shared memory, filled by a
// warp of its own: looking one up takes two dependent loads and five
// divisions (about 2000 cycles), as long as the MMAs of a short tile.
constexpr int kRing = 4;
struct RingSlot {
  int more, f, tile, expert, row0, valid, pad[2];
};

// Waits of a converged warp (every lane polls): false as soon as one lane gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit));
}
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort,
                                                  uint64_t limit) {
  return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort, limit));
}

// The scheduler warp (lane 0): items first, first + step, ... below total, then
// a slot without one.
template <int kRows>
__device__ __forceinline__ void schedule(const MxGemmArgs& args, RingSlot* ring, uint32_t ifull0, uint32_t iempty0,
                                         int first, int step, int total, int num_tiles, int nf, volatile int* abort,
                                         uint64_t limit) {
  int item = first;
  for (int n = 0;; ++n, item += step) {
    const int slot = n % kRing;
    RingSlot v{};
    if (item < total) {
      const Item w = item_of<kRows>(args, item, num_tiles, nf);
      v.more = 1;
      v.f = w.f;
      v.tile = w.tile;
      v.expert = w.expert;
      v.row0 = w.row0;
      v.valid = w.valid;
    }
    if (!mbar_wait(iempty0 + 8 * slot, ((uint32_t)(n / kRing) & 1u) ^ 1u, abort, limit)) {
      *abort = 1;
      atomicOr(args.status, kDevErrTimeout);
      return;
    }
    ring[slot] = v;
    mbar_arrive(ifull0 + 8 * slot);
    if (!v.more) return;
  }
}

// The n-th item, for a converged warp; false when there is none or a wait
// gave up (then *ok is false).
__device__ __forceinline__ bool next_item(const RingSlot* ring, uint32_t ifull0, uint32_t iempty0, int n, Item& w,
                                          bool& ok, volatile int* abort, uint64_t limit) {
  const int slot = n % kRing;
  if (!warp_wait(ifull0 + 8 * slot, (uint32_t)(n / kRing) & 1u, abort, limit)) {
    ok = false;
    return false;
  }
  const RingSlot v = ring[slot];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(iempty0 + 8 * slot);
  w.f = uniform(v.f);
  w.tile = uniform(v.tile);
  w.expert = uniform(v.expert);
  w.row0 = uniform(v.row0);
  w.valid = uniform(v.valid);
  return uniform(v.more) != 0;
}

// silu(g) * u.  exp and the reciprocal without the steps that keep subnormal
// results: 1 + exp is 1 where exp(-g) is one, and a reciprocal that is one
// counts as 0 (g below -87).  The exponent is one rounded product, so silu is
// off by 2^-21 + max(-g, 0) 2^-23 of itself at most: past 2^-20 only below g =
// -4, where silu is under a 50th of |g| and a 4-bit value keeps two bits of it.
// The accurate exponential took 2 to 3 % of a prompt's pass.
__device__ __forceinline__ float swiglu(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.44269504088896f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r * u;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// a = silu(g) * u of 32 neighbouring features of one token, quantised:
// 16 bytes of codes, one scale byte.
__device__ __forceinline__ void store_swiglu_block(const float (&g)[32], float (&u)[32], uint8_t* codes,
                                                   uint8_t* scale) {
  float hi = 0.0f, lo = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    u[i] = swiglu(g[i], u[i]);
    u[i + 1] = swiglu(g[i + 1], u[i + 1]);
    hi = max3(hi, u[i], u[i + 1]);   // NaN if one is
    lo = min3(lo, u[i], u[i + 1]);
  }
  const uint32_t byte = scale_byte(max(__float_as_uint(hi) & 0x7FFFFFFFu, __float_as_uint(lo) & 0x7FFFFFFFu));
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

template <bool kW13, int BN, bool kSwap>
__global__ void __launch_bounds__(kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
                   const __grid_constant__ CUtensorMap x_map_small, const MxGemmArgs args) {
  using C = Cfg<BN, kSwap>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  __shared__ int s_issued;   // operand loads the producer asked for
  __shared__ __align__(8) uint64_t s_ibar[2 * kRing];   // the ring's full, then empty barriers
  __shared__ __align__(16) RingSlot s_ring[kRing];

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* xchg = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);
  const uint32_t full0 = smem_u32(smem + C::kStages * C::kStageBytes + C::kXchgBytes);
  const uint32_t empty0 = full0 + 8 * C::kStages;
  const uint32_t tfull0 = empty0 + 8 * C::kStages;
  const uint32_t tempty0 = tfull0 + 16;
  const uint32_t drain = tempty0 + 16;
  const uint32_t ifull0 = smem_u32(s_ibar), iempty0 = ifull0 + 8 * kRing;

  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
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
    for (int i = 0; i < kRing; ++i) {
      mbar_init(ifull0 + 8 * i, 1);
      mbar_init(iempty0 + 8 * i, 2 + kEpiWarps);
    }
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
  const uint32_t tmem = (uint32_t)uniform((int)s_tmem_base);
  pdl_wait();
  pdl_trigger();
  const int num_tiles =
      uniform(args.identity_T ? (args.identity_T + C::kTokens - 1) / C::kTokens : *args.num_tiles);
  const int total = num_tiles * nf;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol_w = policy_evict_normal();
    const uint64_t pol_x = policy_evict_last();
    const uint32_t s0 = smem_u32(smem);
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;   // loads
    bool ok = true;
    Item w;
    for (int n = 0; ok && next_item(s_ring, ifull0, iempty0, n, w, ok, &s_abort, wlim); ++n) {
      const bool small = kSwap || w.valid <= kSmallRows;   // the token box
      const uint32_t a_tx = (small ? kSmallRows : kMxTileRows) * 128u;
      // scale tiles of B that exist (the last item of an odd number of 128-row tiles has one)
      const int sft0 = w.f * BN / kSfRows;
      const int sft = min(C::kSfbTiles, args.features / kSfRows - sft0);
      const uint8_t* sfa = args.a_sf + (size_t)w.tile * kchunks * kSfChunkBytes;
      const uint8_t* sfb = args.b_sf + ((size_t)w.expert * (args.features / kSfRows) + sft0) * kchunks * kSfChunkBytes;
      for (int ks = 0; ks < ksteps; ++ks) {
        if (!warp_wait(empty0 + 8 * stage, phase ^ 1u, &s_abort, wlim)) {
          ok = false;
          break;
        }
        const uint32_t sA = s0 + stage * C::kStageBytes;
        const uint32_t sB = sA + C::kABytes;
        const uint32_t sFa = sB + C::kBBytes, sFb = sFa + C::kSfaBytes;
        const uint32_t fb = full0 + 8 * stage;
        const uint32_t sf_bytes = (uint32_t)min(2, kchunks - 2 * ks) * kSfChunkBytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(fb, a_tx + C::kBBytes + sf_bytes * (1 + sft));
          if (kW13)
            tma_load_5d(sB, &w_map, ks * 128, 0, 0, w.f * (BN / 64), w.expert, fb, pol_w);
          else
            tma_load_3d(sB, &w_map, ks * 128, w.f * BN, w.expert, fb, pol_w);
          tma_load_2d(sA, small ? &x_map_small : &x_map, ks * 128, w.row0, fb, pol_x);
          bulk_load(sFa, sfa + (size_t)(2 * ks) * kSfChunkBytes, sf_bytes, fb);
          bulk_load(sFb, sfb + (size_t)(2 * ks) * kSfChunkBytes, sf_bytes, fb);
          if (C::kSfbTiles > 1 && sft > 1)
            bulk_load(sFb + 2 * kSfChunkBytes, sfb + ((size_t)kchunks + 2 * ks) * kSfChunkBytes, sf_bytes, fb);
        }
        __syncwarp();
        ++issued;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      s_abort = 1;
      if (lane == 0) atomicOr(args.status, kDevErrTimeout);
    }
    if (lane == 0) s_issued = issued;
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    int stage = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    // descriptors of stage 0, built once; soff is the stage's offset in their 16-byte units
    const uint32_t s0 = smem_u32(smem);
    const uint64_t adesc0 = sdesc_sw128(s0, 16, 1024), bdesc0 = sdesc_sw128(s0 + C::kABytes, 16, 1024);
    const uint64_t fadesc0 = sdesc_scales(s0 + C::kABytes + C::kBBytes);
    const uint64_t fbdesc0 = sdesc_scales(s0 + C::kABytes + C::kBBytes + C::kSfaBytes);
    constexpr int kN = C::kCols;
    constexpr uint32_t kI0 = idesc_mxf4(128, kN, 0), kI1 = idesc_mxf4(128, kN, 1);
    uint32_t soff = 0;
    const bool leader = elect_one();
    Item w;
    for (int n = 0; ok && next_item(s_ring, ifull0, iempty0, n, w, ok, &s_abort, wlim); ++n) {
      // an item narrower than a scale tile takes its columns of it
      const uint32_t sfb_skip = (BN < kSfRows) ? (uint32_t)(w.f * BN % kSfRows) / 32u : 0u;
      if (!warp_wait(tempty0 + 8 * acc, acc_phase ^ 1u, &s_abort, wlim)) {
        ok = false;
        break;
      }
      const uint32_t d0 = tmem + acc * C::kCols;
      // one stage: chunks of 128 elements, for each the scales (A's in columns
      // ta + 4c, those of B's tile t in tb + (c kSfbTiles + t) 4), then two MMAs
      auto step = [&](auto two, bool first, bool last) -> bool {
        if (!mbar_wait(full0 + 8 * stage, phase, &s_abort, wlim)) return false;
        tc_fence_after();
        const uint32_t ta = tmem + C::kSfCol0 + stage * C::kSfCols, tb = ta + 8;
        const uint64_t ad = adesc0 + soff, bd = bdesc0 + soff, fa = fadesc0 + soff, fbd = fbdesc0 + soff;
        const uint32_t done = empty0 + 8 * stage;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
          soff = 0;
        } else {
          soff += C::kStageBytes >> 4;
        }
        if (leader) {
          constexpr int kChunks = decltype(two)::value ? 2 : 1;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            cp_scales(ta + 4 * c, fa + c * kSfUnits);
#pragma unroll
            for (int t = 0; t < C::kSfbTiles; ++t)
              cp_scales(tb + 4 * (c * C::kSfbTiles + t), fbd + (2 * t + c) * kSfUnits);
          }
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const uint32_t sa = ta + 4 * c, sb = tb + 4 * c * C::kSfbTiles + sfb_skip;
            const uint64_t m = (kSwap ? bd : ad) + 4 * c, k = (kSwap ? ad : bd) + 4 * c;
            mma_mxf4(d0, m, k, kI0, kSwap ? sb : sa, kSwap ? sa : sb, (c > 0 || !first) ? 1u : 0u);
            mma_mxf4(d0, m + 2, k + 2, kI1, kSwap ? sb : sa, kSwap ? sa : sb, 1u);
          }
          mma_commit(done);
          if (last) mma_commit(tfull0 + 8 * acc);
        }
        return true;
      };
      for (int ks = 0; ok && ks < kchunks / 2; ++ks) ok = step(std::true_type{}, ks == 0, 2 * ks + 2 == kchunks);
      if (ok && (kchunks & 1)) ok = step(std::false_type{}, kchunks == 1, true);
      ok = __all_sync(0xffffffffu, ok);
      if (++acc == C::kNumAcc) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok) {
      s_abort = 1;
      if (lane == 0) atomicOr(args.status, kDevErrTimeout);
    }
    // all issued MMAs must be complete before TMEM is released
    if (leader) mma_commit(drain);
    __syncwarp();
    volatile int no_abort = 0;
    mbar_wait(drain, 0, &no_abort);
    __syncwarp();
  } else if (warp < kRoleWarps) {
    // ------------------------------------------------------------ scheduler
    if (warp == 2 && lane == 0)
      schedule<C::kTokens>(args, s_ring, ifull0, iempty0, blockIdx.x, gridDim.x, total, num_tiles, nf, &s_abort, wlim);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;              // TMEM lanes this warp may access
    const int half = (warp - kRoleWarps) / 4;  // which blocks of columns
    const int r = quarter * 32 + lane;         // token row of the tile (swapped: weight row of the item)
    constexpr int kBlockCols = kW13 ? 64 : 32; // columns of one block (W13: 32 gate, 32 up)
    constexpr int kBlocks = BN / kBlockCols;
    int acc = 0;
    uint32_t acc_phase = 0;
    Item w;
    bool ok = true;
    for (int n = 0;; ++n) {
      bool got = next_item(s_ring, ifull0, iempty0, n, w, ok, &s_abort, wlim);
      const bool more = got || !ok;
      if (got) got = warp_wait(tfull0 + 8 * acc, acc_phase, &s_abort, wlim);
      if (more && !got) ok = false;
      // a gate warp and its up warp go on or stop together (they meet on a barrier for every item)
      const int pair = 1 + half * 2 + quarter / 2;
      if (kSwap && kW13) got = bar_and(pair, 64, got);
      if (!got) break;
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(quarter * 32) << 16) + acc * C::kCols;
      if (kSwap) {
        // lane: weight row; columns: tokens, 16 of them this warp's
        float v[16];
        const int t0 = half * 16;
        if (t0 < w.valid) tmem_load16(tbase + t0, v);
        if (kW13) {
          // the item's rows are 32 gate, 32 up, 32 gate, 32 up features: quarters 1 and 3 hand
          // theirs over; a block of 32 features lies across the lanes of a gate warp
          float* buf = xchg + (half * 2 + quarter / 2) * (16 * 32) + lane;
          if (quarter & 1) {
#pragma unroll
            for (int j = 0; j < 16; ++j) buf[j * 32] = v[j];
          }
          bar_sync(pair, 64);
          if (!(quarter & 1)) {
            const int feat = w.f * (BN / 2) + (quarter / 2) * 32;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              if (t0 + j >= w.valid) break;
              const float a = swiglu(v[j], buf[j * 32]);
              const uint32_t byte = scale_byte(__float_as_uint(warp_amax(a)) & 0x7FFFFFFFu);
              const float x = byte == 255u ? 0.0f : a * scale_inverse(byte);
              const float y = __shfl_down_sync(0xffffffffu, x, 1);
              const size_t row = (size_t)w.row0 + t0 + j;
              if (!(lane & 1)) args.out_codes[(row * args.out_ld + feat + lane) / 2] = (uint8_t)pack2(x, y);
              if (lane == 0)
                args.out_sf[((size_t)w.tile * (args.out_ld / kSfChunkK) + feat / kSfChunkK) * kSfChunkBytes +
                            sf_row_offset(t0 + j) + (feat % kSfChunkK) / kBlock] = (uint8_t)byte;
            }
          }
          bar_sync(pair, 64);   // the buffer is free again
        } else {
          const int feat = w.f * BN + r;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (t0 + j < w.valid)
              args.out[((size_t)w.row0 + t0 + j) * args.out_ld + feat] =
                  __bfloat16_as_ushort(__float2bfloat16_rn(v[j]));
        }
      } else if (quarter * 32 < w.valid) {
        const size_t row = (size_t)w.row0 + r;
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
    if (!ok) {
      s_abort = 1;
      if (lane == 0) atomicOr(args.status, kDevErrTimeout);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
  if (threadIdx.x == 0 && s_abort) land_loads(full0, C::kStages, s_issued);
}

// ------------------------------------------------------------------ CTA pairs
// The same GEMMs on pairs of CTAs (a cluster of two on two SMs, one
// cta_group::2 MMA of 256 token rows x 192 weight rows): each CTA loads its
// own 128 token rows and half of the weight rows and holds the result of its
// 128 rows.  192 columns, because two accumulators and the scale columns then
// fit into TMEM: with 256 the accumulators have to share columns, and each
// tile's first MMA waits for the last one's epilogue to begin (about 1800
// cycles, where a tile of K = 768 has 1700 cycles of MMAs).  What holds a tile
// back, from copies of the kernel timed without a part (8192 tokens x 8 of 128
// experts | 4096 x 2 of 8, a whole pass of 190 | 490 us): operand loads cut to
// 8 rows 171 | 415, without the scale copies 5 | 19 less, W13's epilogue 5 less,
// W2's output not written 33 | 14 less; and an expert's last tile is half empty
// on average (320 tiles where 256 would be full | 36 where 32).
//
// TMEM (512 columns): accumulators at 0 and 192, five slots of scale columns
// behind them.  W13's shared memory holds two stages more than there are slots:
// a slot is rewritten once the commit of the step that used it last has arrived.
//
// Twelve epilogue warps, one per lane quarter and 64-column block.  W2 rows
// leave through shared memory as 32-row x 64-column tiled stores (a lane's
// direct 16-byte stores touch one line per row); a lane quarter with padding
// rows stores directly, so that padding is never written.
constexpr int kPairRowsMx = 2 * kMxTileRows;
constexpr int kPairN = 192;
constexpr int kPairEpiWarps = 12;
constexpr int kPairThreads = (kRoleWarps + kPairEpiWarps) * 32;
constexpr int kSfSlots = 5;

template <bool kW13>
struct PairCfgMx {
  static constexpr uint32_t kABytes = kMxTileRows * 128;
  static constexpr uint32_t kBBytes = (kPairN / 2) * 128;
  static constexpr uint32_t kSfaBytes = 2 * kSfChunkBytes;
  static constexpr uint32_t kSfbBytes = 2 * 2 * kSfChunkBytes;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  static constexpr uint32_t kOutBytes = kW13 ? 0 : kPairEpiWarps * 32 * 128;
  static constexpr uint32_t kBarBytes = 512;
  static constexpr int kStages = kW13 ? 7 : 5;
  static constexpr uint32_t kSmemBytes = kStages * kStageBytes + kOutBytes + kBarBytes + 1024;
  static constexpr uint32_t kSfCols = 24;
  static constexpr uint32_t kSfCol0 = 2 * kPairN;
  static_assert(kSmemBytes <= kSmemLimit, "stages fit");
  static_assert(kSfCol0 + kSfSlots * kSfCols <= 512, "accumulators and scales fit in TMEM");
  static_assert(kStageBytes % 1024 == 0, "stages stay aligned to the swizzle atom");
};

template <bool kW13>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    mx_gemm_pair_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
                        const __grid_constant__ CUtensorMap sfa_map, const __grid_constant__ CUtensorMap sfb_map,
                        const __grid_constant__ CUtensorMap y_map, const MxGemmArgs args) {
  using C = PairCfgMx<kW13>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  __shared__ int s_issued;   // operand loads the producer asked for
  __shared__ volatile PairEnd s_peer;
  __shared__ __align__(8) uint64_t s_ibar[2 * kRing];   // the ring's full, then empty barriers
  __shared__ __align__(16) RingSlot s_ring[kRing];

  const uint32_t rank = cluster_ctarank();   // 0: issues the MMAs
  const bool lead = rank == 0;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_out = smem + C::kStages * C::kStageBytes;
  const uint32_t full0 = smem_u32(s_out + C::kOutBytes);
  const uint32_t empty0 = full0 + 8 * C::kStages;
  const uint32_t tfull0 = empty0 + 8 * C::kStages;
  const uint32_t tempty0 = tfull0 + 16;
  const uint32_t drain = tempty0 + 16;
  const uint32_t ifull0 = smem_u32(s_ibar), iempty0 = ifull0 + 8 * kRing;

  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  const int kchunks = args.K / kSfChunkK;
  const int ksteps = (args.K + kStageK - 1) / kStageK;
  const int nf = (args.features + kPairN - 1) / kPairN;
  const int pair0 = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
  const uint64_t wlim = args.wait_ns ? args.wait_ns : kWaitLimitNs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 2 * kPairEpiWarps);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(ifull0 + 8 * i, 1);
      mbar_init(iempty0 + 8 * i, (lead ? 2 : 1) + kPairEpiWarps);
    }
    s_abort = 0;
    s_peer.gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&s_tmem_base), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&w_map);
    prefetch_tmap(&x_map);
    prefetch_tmap(&sfa_map);
    prefetch_tmap(&sfb_map);
    if (!kW13) prefetch_tmap(&y_map);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)s_tmem_base);
  pdl_wait();
  pdl_trigger();
  const int num_tiles =
      uniform(args.identity_T ? (args.identity_T + kPairRowsMx - 1) / kPairRowsMx : *args.num_tiles);
  const int total = num_tiles * nf;

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    const uint64_t pol_w = policy_evict_normal();
    const uint64_t pol_x = policy_evict_last();
    const uint32_t s0 = smem_u32(smem);
    const int me = uniform((int)rank);
    const uint32_t full_lead = mapa_shared(full0, 0);   // the even CTA's full barriers
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;   // loads
    bool ok = true;
    Item w;
    for (int n = 0; ok && next_item(s_ring, ifull0, iempty0, n, w, ok, &s_abort, wlim); ++n) {
      const int arow = w.row0 + me * kMxTileRows;
      const int sfa_row = (2 * w.tile + me) * kchunks;
      // the 128-row scale tiles that hold the item's rows (from the middle of
      // the first one on for an odd item)
      const int sfb_row = (w.expert * (args.features / kSfRows) + w.f * kPairN / kSfRows) * kchunks;
      for (int ks = 0; ks < ksteps; ++ks) {
        if (!warp_wait_cluster(empty0 + 8 * stage, phase ^ 1u, &s_abort, wlim)) {
          ok = false;
          break;
        }
        const uint32_t sA = s0 + stage * C::kStageBytes;
        const uint32_t sB = sA + C::kABytes;
        const uint32_t sFa = sB + C::kBBytes, sFb = sFa + C::kSfaBytes;
        const uint32_t fb = full_lead + 8 * stage;
        if (elect_one()) {
          if (lead) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * C::kStageBytes);
          if (kW13) {
            // 96 of the item's 192 rows: three runs of 32, gate and up in turns
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const int run = 3 * me + i;
              tma_load_5d_pair(sB + i * 32 * 128, &w_map, ks * 128, 0, run & 1, w.f * 3 + (run >> 1), w.expert, fb, pol_w);
            }
          } else {
            tma_load_3d_pair(sB, &w_map, ks * 128, w.f * kPairN + me * (kPairN / 2), w.expert, fb, pol_w);
          }
          tma_load_2d_pair(sA, &x_map, ks * 128, arow, fb, pol_x);
          // scale chunks of this stage's 256 elements (a last odd chunk brings its
          // neighbour's along; the MMAs stop at K)
          tma_load_2d_pair(sFa, &sfa_map, 0, sfa_row + 2 * ks, fb, pol_x);
          tma_load_2d_pair(sFb, &sfb_map, 0, sfb_row + 2 * ks, fb, pol_w);
          tma_load_2d_pair(sFb + 2 * kSfChunkBytes, &sfb_map, 0, sfb_row + kchunks + 2 * ks, fb, pol_w);
        }
        __syncwarp();
        ++issued;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      s_abort = 1;
      if (lane == 0) atomicOr(args.status, kDevErrTimeout);
    }
    if (lane == 0) s_issued = issued;
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lead) {
      int stage = 0;
      uint32_t phase = 0;
      int old = 0;                   // the stage of the step kSfSlots before the next one
      uint32_t old_phase = 0;
      int slot = 0, steps = 0;
      const uint32_t s0 = smem_u32(smem);
      const uint64_t adesc0 = sdesc_sw128(s0, 16, 1024), bdesc0 = sdesc_sw128(s0 + C::kABytes, 16, 1024);
      const uint64_t fadesc0 = sdesc_scales(s0 + C::kABytes + C::kBBytes);
      const uint64_t fbdesc0 = sdesc_scales(s0 + C::kABytes + C::kBBytes + C::kSfaBytes);
      constexpr uint32_t kI0 = idesc_mxf4(kPairRowsMx, kPairN, 0), kI1 = idesc_mxf4(kPairRowsMx, kPairN, 1);
      uint32_t soff = 0;
      const bool leader = elect_one();
      bool ok = true;
      Item w;
      for (int n = 0; ok && next_item(s_ring, ifull0, iempty0, n, w, ok, &s_abort, wlim); ++n) {
        const int acc = n & 1;
        const uint32_t sfb_skip = (uint32_t)(w.f * kPairN % kSfRows) / 32u;
        if (!warp_wait_cluster(tempty0 + 8 * acc, ((uint32_t)(n >> 1) & 1u) ^ 1u, &s_abort, wlim)) {
          ok = false;
          break;
        }
        const uint32_t d0 = tmem + acc * kPairN;
        auto step = [&](auto two, bool first, bool last) -> bool {
          if (!mbar_wait_cluster(full0 + 8 * stage, phase, &s_abort, wlim)) return false;
          // the scale slot is free once the step kSfSlots before this one has been committed
          if (C::kStages > kSfSlots && steps >= kSfSlots &&
              !mbar_wait_cluster(empty0 + 8 * old, old_phase, &s_abort, wlim))
            return false;
          tc_fence_after();
          const uint32_t ta = tmem + C::kSfCol0 + slot * C::kSfCols, tb = ta + 8;
          const uint64_t ad = adesc0 + soff, bd = bdesc0 + soff, fa = fadesc0 + soff, fbd = fbdesc0 + soff;
          const uint32_t done = empty0 + 8 * stage;
          if (++slot == kSfSlots) slot = 0;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
            soff = 0;
          } else {
            soff += C::kStageBytes >> 4;
          }
          if (++steps > kSfSlots && ++old == C::kStages) {
            old = 0;
            old_phase ^= 1u;
          }
          if (leader) {
            constexpr int kChunks = decltype(two)::value ? 2 : 1;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              cp_scales_pair(ta + 4 * c, fa + c * kSfUnits);
              cp_scales_pair(tb + 8 * c, fbd + c * kSfUnits);
              cp_scales_pair(tb + 8 * c + 4, fbd + (2 + c) * kSfUnits);
            }
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              const uint32_t sb = tb + 8 * c + sfb_skip;
              mma_mxf4_pair(d0, ad + 4 * c, bd + 4 * c, kI0, ta + 4 * c, sb, (c > 0 || !first) ? 1u : 0u);
              mma_mxf4_pair(d0, ad + 4 * c + 2, bd + 4 * c + 2, kI1, ta + 4 * c, sb, 1u);
            }
            mma_commit_pair(done, 0x3);
            if (last) mma_commit_pair(tfull0 + 8 * acc, 0x3);
          }
          return true;
        };
        for (int ks = 0; ok && ks < kchunks / 2; ++ks) ok = step(std::true_type{}, ks == 0, 2 * ks + 2 == kchunks);
        if (ok && (kchunks & 1)) ok = step(std::false_type{}, kchunks == 1, true);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (!ok) {
        s_abort = 1;
        if (lane == 0) atomicOr(args.status, kDevErrTimeout);
      }
      if (leader) mma_commit_pair(drain, 0x3);
      __syncwarp();
      volatile int no_abort = 0;
      mbar_wait(drain, 0, &no_abort);
    }
    __syncwarp();
  } else if (warp < kRoleWarps) {
    // ------------------------------------------------------------ scheduler (both CTAs)
    if (warp == 2 && lane == 0)
      schedule<kPairRowsMx>(args, s_ring, ifull0, iempty0, pair0, pairs, total, num_tiles, nf, &s_abort, wlim);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;              // TMEM lanes this warp may access
    const int b = (warp - kRoleWarps) / 4;     // its 64-column block
    const int r = quarter * 32 + lane;         // token row of the CTA's 128
    uint8_t* buf = s_out + (warp - kRoleWarps) * (32 * 128);
    const uint32_t sbuf = smem_u32(buf);
    Item w;
    bool ok = true;
    for (int n = 0; next_item(s_ring, ifull0, iempty0, n, w, ok, &s_abort, wlim); ++n) {
      const int acc = n & 1;
      int got = 1;
      if (lane == 0) got = mbar_wait_cluster(tfull0 + 8 * acc, (uint32_t)(n >> 1) & 1u, &s_abort, wlim) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (!got) {
        if (lane == 0) {
          s_abort = 1;
          atomicOr(args.status, kDevErrTimeout);
        }
        break;
      }
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(quarter * 32) << 16) + acc * kPairN + b * 64;
      const int valid = w.valid - (int)rank * kMxTileRows;       // of this CTA's rows
      const size_t row = (size_t)w.row0 + rank * kMxTileRows + r;
      // weight rows past an expert's last (the last item of it) are not stored
      const bool work = quarter * 32 < valid && w.f * kPairN + b * 64 < args.features;
      float p[32], q[32];
      if (work) tmem_load32x2(tbase, p, tbase + 32, q);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(mapa_shared(tempty0 + 8 * acc, 0));
      if (!work) continue;
      if (kW13) {
        const int feat = w.f * (kPairN / 2) + b * 32;
        if (r < valid)
          store_swiglu_block(p, q, args.out_codes + (row * args.out_ld + feat) / 2,
                             args.out_sf +
                                 ((size_t)(2 * w.tile + rank) * (args.out_ld / kSfChunkK) + feat / kSfChunkK) * kSfChunkBytes +
                                 sf_row_offset(r) + (feat % kSfChunkK) / kBlock);
      } else {
        const int feat = w.f * kPairN + b * 64;
        if (quarter * 32 + 32 <= valid) {
          // 128 bytes a row in the 128-byte swizzle: 16-byte piece j of row l at j ^ (l & 7)
          if (lane == 0) tma_store_wait_read();
          __syncwarp();
          auto pieces = [&](const float (&v)[32], int j0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 x = __floats2bfloat162_rn(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
                o[e] = *reinterpret_cast<const uint32_t*>(&x);
              }
              *reinterpret_cast<uint4*>(buf + lane * 128 + (((j0 + j) ^ (lane & 7)) * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          };
          pieces(p, 0);
          pieces(q, 4);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tma_store_2d(&y_map, sbuf, feat, w.row0 + (int)rank * kMxTileRows + quarter * 32);
        } else if (r < valid) {
          store_bf16_block(p, args.out + row * args.out_ld + feat);
          store_bf16_block(q, args.out + row * args.out_ld + feat + 32);
        }
      }
    }
    if (!ok) {
      s_abort = 1;
      if (lane == 0) atomicOr(args.status, kDevErrTimeout);
    }
    if (!kW13 && lane == 0) tma_store_wait();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  end_pair(lead, full0, drain, C::kStages, s_issued, s_abort, &s_peer, [](int) { return C::kStageBytes; });
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// Pairs of CTAs that can be resident at once, looked up once per device and kernel.
template <bool kW13>
int resident_pairs_mx(int sms) {
  static int cache[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)(sms / 2), 1, 1);
  cfg.blockDim = dim3(kPairThreads, 1, 1);
  cfg.dynamicSmemBytes = PairCfgMx<kW13>::kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, mx_gemm_pair_kernel<kW13>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = sms / 2;
  }
  n = n < sms / 2 ? n : sms / 2;
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

template <bool kW13>
void launch_pair_mx(const MxMaps& m, MxGemmArgs a, int64_t max_tiles, int sms, cudaStream_t s) {
  auto kernel = mx_gemm_pair_kernel<kW13>;
  constexpr int smem = (int)PairCfgMx<kW13>::kSmemBytes;
  static bool attr_set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int64_t items = max_tiles * ((a.features + kPairN - 1) / kPairN);
  if (items <= 0) return;
  const int cap = resident_pairs_mx<kW13>(sms);
  const int pairs = (int)(items < cap ? items : cap);
  a.concurrent = pairs;
  launch_pdl(kernel, dim3(2 * pairs), dim3(kPairThreads), smem, s, m.w, m.x, m.sfa, m.sfb, m.y, a);
}

template <bool kW13, int BN, bool kSwap>
void launch(const MxMaps& m, MxGemmArgs a, int64_t max_tiles, int sms, cudaStream_t s) {
  auto kernel = mx_gemm_kernel<kW13, BN, kSwap>;
  constexpr int smem = (int)Cfg<BN, kSwap>::kSmemBytes;
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
  launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, s, m.w, m.x, m.x_small, a);
}

// ------------------------------------------------------------------ front
// One launch before the GEMMs: the tile list, and the activations in tile
// order (codes of the routed rows, and scales in the chunks that the MMAs
// take).  Bound by memory (the codes once more in L2) and by chains of
// dependent loads, so CTAs work side by side on parts that need little of each
// other: CTA 0 writes the list; the next ones place scales, each deriving the
// experts' segments from the block list on its own; the next copy codes,
// which lie in the order of the routes and need no list; and where the GEMMs
// are bound by the weights' bytes, the last ones ask for W13's first.  With identity_T
// there is no list and the codes stay where they are.  8192 tokens x 8 of 128
// experts, H 2048: 20 us for 137 MB through L2 (37 with a CTA to each tile for
// codes and scales); 4096 x 2 of 8, H 4096: 8 us (40); one token: 4 us (7).
constexpr int kFrontThreads = 256;
constexpr int kFrontWarps = kFrontThreads / 32;
constexpr int kFrontChunks = 16;   // scale chunks of a tile placed at once
constexpr int kFrontRows = 4;      // code rows a warp copies at once
// About what HBM delivers while the front runs (more delays W13's own loads).
// One token on 2 of 8 experts, H 4096, I 14336 | 512 tokens x 8 of 128, H 2048,
// I 768: none 44.0 | 68.4 us a pass; 16 MB 41.9 | 67.4, 24 MB 41.8 | 66.8, 32 MB
// 42.6 | 67.1, 48 MB 44.0 | 66.7.  Spread over every SM: requests queue in the
// copy engine that W13's loads pass through (H 7168, 48 MB from 28 SMs: 44 -> 58).
constexpr int kPrefetchBytes = 24 << 20, kPrefetchPiece = 4096, kPrefetchParts = 4;

// Codes of padded rows [0, P) (zeros in a row without a route), kFrontRows rows
// a warp, two 16-byte pieces a lane of each; the next rows' routes are under
// way meanwhile.
__device__ __forceinline__ void front_codes(const MxFrontArgs& a, int first, int step, int lane) {
  const int R = (int)min((long long)a.T * a.slots, 0x7FFFFFFFll), pieces = a.H / 32;
  auto route_at = [&](long long row) { return lane < kFrontRows && row + lane < a.max_rows ? a.sorted[row + lane] : -1; };
  long long row0 = (long long)first * kFrontRows;
  int id = route_at(row0);
  const int P = *a.num_padded;
  if (P < 0 || P > a.max_rows) return;
  while (row0 < P) {
    const long long next = row0 + (long long)step * kFrontRows;
    const int id_next = route_at(next);
    const int token = id >= 0 && id < R ? id / a.slots : -1;
    int tok[kFrontRows];
#pragma unroll
    for (int j = 0; j < kFrontRows; ++j) tok[j] = __shfl_sync(0xffffffffu, token, j);
    for (int p0 = lane; p0 < pieces; p0 += 64) {
      uint4 v[kFrontRows][2];
#pragma unroll
      for (int j = 0; j < kFrontRows; ++j) {
        const uint4* src = reinterpret_cast<const uint4*>(a.codes + (size_t)max(tok[j], 0) * (a.H / 2));
#pragma unroll
        for (int u = 0; u < 2; ++u)
          v[j][u] = tok[j] >= 0 && p0 + 32 * u < pieces ? __ldg(src + p0 + 32 * u) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kFrontRows; ++j) {
        uint4* dst = reinterpret_cast<uint4*>(a.x_perm + (size_t)(row0 + j) * (a.H / 2));
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (row0 + j < P && p0 + 32 * u < pieces) dst[p0 + 32 * u] = v[j][u];
      }
    }
    row0 = next;
    id = id_next;
  }
}

// The codes that W13's first items read, into L2: units of 32 gate and the same
// 32 up features, of the experts in the order of the list.
__device__ __forceinline__ void front_prefetch(const MxFrontArgs& a, int first, int step, int lane) {
  const int P = *a.num_padded;
  if (P < 0 || P > a.max_rows) return;
  const int nb = P / a.B, per = a.I / 32;
  const size_t row = a.H / 2;
  for (int i = first; i < a.prefetch_units * kPrefetchParts; i += step) {
    const int unit = i / kPrefetchParts, part = i % kPrefetchParts;
    int skip = unit / per, expert = -1;   // the expert: that many before it in the list
    for (int b0 = 0; b0 < nb && expert < 0; b0 += 32) {
      const int b = b0 + lane;
      const int e = b < nb ? a.block_expert[b] : -1, prev = b < nb && b ? a.block_expert[b - 1] : -1;
      uint32_t heads = __ballot_sync(0xffffffffu, b < nb && e != prev);
      const int n = __popc(heads);
      if (skip < n) {
        for (int j = 0; j < skip; ++j) heads &= heads - 1;
        expert = __shfl_sync(0xffffffffu, e, __ffs(heads) - 1);
        break;
      }
      skip -= n;
    }
    if (expert < 0 || expert >= a.N) return;
    // 32 rows are contiguous
    const int bytes = 32 / kPrefetchParts * (int)row;
    const uint8_t* gate = a.w13 + ((size_t)expert * 2 * a.I + (unit % per) * 32) * row + part * bytes;
    for (int p = lane * kPrefetchPiece; p < bytes; p += 32 * kPrefetchPiece) {
      const uint32_t n = (uint32_t)min(kPrefetchPiece, bytes - p);
      bulk_prefetch(gate + p, n);
      bulk_prefetch(gate + (size_t)a.I * row + p, n);
    }
  }
}

__global__ void __launch_bounds__(kFrontThreads) mx_front_kernel(const MxFrontArgs a) {
  __shared__ int s_first[256], s_last[256], s_used[256], s_off[257], s_scan[kFrontWarps];
  __shared__ int s_bad;
  __shared__ int s_token[kMxTileRows];
  __shared__ __align__(16) uint32_t s_sf[kFrontChunks * (kSfChunkBytes / 4)];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x > a.scale_ctas) {
    const int cta = (int)blockIdx.x - 1 - a.scale_ctas;
    const int prefetch_ctas = (int)gridDim.x - 1 - a.scale_ctas - a.code_ctas;
    if (cta < a.code_ctas)
      front_codes(a, cta * kFrontWarps + warp, a.code_ctas * kFrontWarps, lane);
    else
      front_prefetch(a, cta - a.code_ctas + warp * prefetch_ctas,
                     prefetch_ctas * kFrontWarps, lane);
    return;
  }
  const int sub_rows = min(a.tile_rows, kMxTileRows);   // rows of a scale tile
  const int subs = a.tile_rows / sub_rows;
  const int kchunks = a.H / kSfChunkK;
  const long long R = (long long)a.T * a.slots;
  int total;   // tiles
  if (a.identity_T) {
    if (blockIdx.x == 0) return;
    total = (a.identity_T + a.tile_rows - 1) / a.tile_rows;
  } else {
    const int P = *a.num_padded;
    const bool bad_count = P < 0 || (long long)P > a.max_rows || P % a.B != 0;
    const int nb = bad_count ? 0 : P / a.B;
    s_first[tid] = 0;
    s_last[tid] = 0;
    if (tid == 0) s_bad = bad_count ? 1 : 0;
    __syncthreads();
    // where each expert's blocks begin and end; a list out of order or range is refused
    auto visit = [&](int b, int prev, int e) {
      if (e < 0 || e >= a.N || prev > e) {
        s_bad = 1;
        return;
      }
      if (prev != e) {
        s_first[e] = b;
        if (prev >= 0) s_last[prev] = b;   // at b = 0: -1
      }
      if (b == nb - 1) s_last[e] = nb;
    };
    constexpr int kUnroll = 4;
    for (int g0 = tid; g0 < nb / 4; g0 += kUnroll * kFrontThreads) {   // four blocks a load
      int4 e[kUnroll];
      int prev[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int g = min(g0 + j * kFrontThreads, nb / 4 - 1);
        e[j] = reinterpret_cast<const int4*>(a.block_expert)[g];
        prev[j] = g ? a.block_expert[4 * g - 1] : -1;
      }
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) {
        const int b = 4 * (g0 + j * kFrontThreads);
        if (b >= nb / 4 * 4) continue;
        visit(b, prev[j], e[j].x);
        visit(b + 1, e[j].x, e[j].y);
        visit(b + 2, e[j].y, e[j].z);
        visit(b + 3, e[j].z, e[j].w);
      }
    }
    if (tid < nb % 4) {
      const int b = nb / 4 * 4 + tid;
      visit(b, b ? a.block_expert[b - 1] : -1, a.block_expert[b]);
    }
    __syncthreads();
    if (s_bad) {
      if (blockIdx.x == 0 && tid == 0) {
        *a.num_tiles = 0;
        atomicOr(a.status, kDevErrBadBlocks);
      }
      return;
    }
    // Rows up to each segment's last route (the padding trails it).  The list
    // needs them, and where a tile is shorter than a block so does every CTA:
    // a block's last tiles may then hold no route, and are left out.
    const int rows = (s_last[tid] - s_first[tid]) * a.B;
    const bool short_tiles = a.tile_rows < a.B;
    if (short_tiles || blockIdx.x == 0) {
      s_used[tid] = 0;
      __syncthreads();
      constexpr int kLoads = 8;
      for (int i0 = tid; i0 < a.N * a.B; i0 += kLoads * kFrontThreads) {   // the last blocks, flattened
        int e[kLoads], row[kLoads], id[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const int i = i0 + j * kFrontThreads;
          e[j] = min(i / a.B, a.N - 1);
          row[j] = (s_last[e[j]] - 1) * a.B + i % a.B;
          id[j] = i < a.N * a.B && s_last[e[j]] > 0 ? a.sorted[row[j]] : -1;
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
          if (id[j] >= 0 && id[j] < R) atomicMax(&s_used[e[j]], row[j] + 1 - s_first[e[j]] * a.B);
      }
      __syncthreads();
      int used = s_used[tid];
      if (used == 0 && rows > 0) {   // a caller's list may end in blocks without a route
        for (used = rows - a.B; used > 0; --used) {
          const int id = a.sorted[s_first[tid] * a.B + used - 1];
          if (id >= 0 && id < R) break;
        }
        s_used[tid] = max(used, 0);
      }
      __syncthreads();
    }
    // tiles of each expert, their exclusive sum
    const int nt = segment_tiles(short_tiles ? s_used[tid] : rows, a.tile_rows);
    int incl = nt;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    int base = 0;
    for (int i = 0; i < warp; ++i) base += s_scan[i];
    s_off[tid] = base + incl - nt;
    if (tid == kFrontThreads - 1) s_off[256] = base + incl;
    __syncthreads();
    total = s_off[256];
    if (blockIdx.x == 0) {
      const int row0 = s_first[tid] * a.B, used = s_used[tid];
      for (int j = 0; j < nt; ++j) {
        const int i = s_off[tid] + j;
        if (i < a.max_tiles) a.tiles[i] = segment_tile(tid, row0, rows, used, a.tile_rows, nt, j, s_off[tid]);
      }
      if (tid == 0) *a.num_tiles = min(total, (int)a.max_tiles);
      return;
    }
  }
  // scales: kFrontChunks chunks of a 128-row tile at a time, through shared memory
  total = min(total, (int)a.max_tiles);
  const int parts = (kchunks + kFrontChunks - 1) / kFrontChunks;
  for (long long unit = (int)blockIdx.x - 1; unit < (long long)total * subs * parts; unit += a.scale_ctas) {
    const long long sub = unit / parts;
    const int c0 = (int)(unit % parts) * kFrontChunks, nc = min(kFrontChunks, kchunks - c0);
    long long row0;
    int rows;
    if (a.identity_T) {
      row0 = sub * sub_rows;
      rows = (int)min((long long)sub_rows, a.identity_T - row0);
    } else {
      const int tile = (int)(sub / subs);
      int lo = 0, hi = a.N - 1;   // the expert: the last whose tiles begin at or before this one
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_off[mid] <= tile) lo = mid;
        else hi = mid - 1;
      }
      row0 = (long long)s_first[lo] * a.B + (long long)(tile - s_off[lo]) * a.tile_rows + (sub % subs) * sub_rows;
      rows = (int)max(0ll, min((long long)sub_rows, (long long)s_last[lo] * a.B - row0));
    }
    if (tid < sub_rows) {
      int token = -1;
      if (tid < rows) {
        if (a.identity_T) {
          token = (int)(row0 + tid);
        } else {
          const int id = a.sorted[row0 + tid];
          if (id >= 0 && id < R) token = id / a.slots;
        }
      }
      s_token[tid] = token;
    }
    __syncthreads();   // also: the last unit's scales are read
    constexpr int kWords = kMxTileRows * kFrontChunks / kFrontThreads;   // words a thread, one chunk of a row each
    uint32_t v[kWords];
    const int c = tid % kFrontChunks;
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const int row = tid / kFrontChunks + j * (kFrontThreads / kFrontChunks);
      const int token = row < sub_rows ? s_token[row] : -1;
      v[j] = token >= 0 && c < nc
                 ? __ldg(reinterpret_cast<const uint32_t*>(a.scales + (size_t)token * (a.H / kBlock)) + c0 + c) : 0u;
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const int row = tid / kFrontChunks + j * (kFrontThreads / kFrontChunks);
      s_sf[(c * kSfChunkBytes + sf_row_offset(row)) / 4] = v[j];
    }
    __syncthreads();
    uint4* out = reinterpret_cast<uint4*>(a.x_sf + ((size_t)sub * kchunks + c0) * kSfChunkBytes);
    for (int i = tid; i < nc * (int)(kSfChunkBytes / 16); i += kFrontThreads)
      out[i] = reinterpret_cast<const uint4*>(s_sf)[i];
  }
}

}  // namespace

bool mx_gemm_smem_ok() {
  int dev = 0, optin = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  return optin >= (int)kSmemLimit;
}

int64_t mx_swap_max_rows(int experts) { return (int64_t)kSwapMaxRows * experts; }

int mx_tile_rows(int64_t rows, int experts) {
  if (rows >= (int64_t)kPairMinRows * experts) return kPairRowsMx;
  return rows <= mx_swap_max_rows(experts) ? kSmallRows : kMxTileRows;
}

int mx_tile_features(int tile_rows, int features, int64_t tiles, int sms) {
  if (tile_rows == kPairRowsMx) return kPairN;
  if (tile_rows == kSmallRows) return 128;
  for (int f = 256; f > 64; f /= 2)
    if (tiles * ((features + f - 1) / f) >= kMinWaves * sms) return f;
  return 64;
}

void launch_mx_gemm(bool w13, const MxMaps& m, const MxGemmArgs& a, int64_t max_tiles, int sms, cudaStream_t s) {
  auto go = [&](auto first, auto second) { (w13 ? first : second)(m, a, max_tiles, sms, s); };
  if (a.tile_rows == kPairRowsMx)
    go(launch_pair_mx<true>, launch_pair_mx<false>);
  else if (a.tile_rows == kSmallRows)
    go(launch<true, 128, true>, launch<false, 128, true>);
  else if (a.tile_features == 256)
    go(launch<true, 256, false>, launch<false, 256, false>);
  else if (a.tile_features == 128)
    go(launch<true, 128, false>, launch<false, 128, false>);
  else
    go(launch<true, 64, false>, launch<false, 64, false>);
}

void launch_mx_front(const MxFrontArgs& args, int sms, cudaStream_t s) {
  // at most two CTAs an SM for the scales and three for the codes: all resident at once
  MxFrontArgs a = args;
  const int64_t subs = a.max_tiles * (a.tile_rows > kMxTileRows ? a.tile_rows / kMxTileRows : 1);
  const int64_t units = subs * ((a.H / kSfChunkK + kFrontChunks - 1) / kFrontChunks);
  const int64_t copies = a.identity_T ? 0 : (a.max_rows + kFrontWarps * kFrontRows - 1) / (kFrontWarps * kFrontRows);
  a.scale_ctas = (int)std::min<int64_t>(units, 2 * sms);
  a.code_ctas = (int)std::min<int64_t>(copies, 3 * sms - 1);
  // where the GEMMs are bound by the weights' bytes
  a.prefetch_units = a.identity_T || a.tile_rows > kMxTileRows ? 0 : kPrefetchBytes / (32 * a.H);
  const int prefetch_ctas = std::min(a.prefetch_units * kPrefetchParts, sms);
  launch_pdl(mx_front_kernel, dim3((unsigned)(1 + a.scale_ctas + a.code_ctas + prefetch_ctas)), dim3(kFrontThreads), 0, s, a);
}

}  // namespace moe
