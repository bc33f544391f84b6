// Products grouped by expert (ragged row counts) and the weight gradient, on
// CTA pairs of the 5th-generation tensor cores:
//   y[p] = x[row(p)] . W_e      (or . W_e^T)          for every row p of expert e
//   dW_e = sum over its rows of x[row(p)]^T dy[row(p)]  (+ add_e)
// row(p) is p, or for a gathered operand the token of route ids[p].
//
// Both are tiles of 256 x 256 on a cluster of two CTAs (tcgen05 cta_group::2,
// M = 256, K = 16 a step, 64 a stage); each CTA holds half of the rows of A
// and of B in its shared memory and half of the sums in its tensor memory.
//   product:  A = 256 output features of W_e (K rows of features, MN-major; its
//             transpose, features of K: K-major), B = up to 256 rows of x
//             (K-major).  The MMA's N is the tile's rows rounded up to 32:
//             columns of an MMA are independent sums over the same K steps, so
//             a row's bits depend neither on N nor on the batch.
//   gradient: A = 256 columns of x, B = 256 columns of dy, both MN-major, K
//             the expert's rows in ascending order.
// Rows gathered by route come by TMA gather4 (four rows a request, one request
// a lane), straight from the token tensor: no copy in segment order.  A row
// index outside the tensor reads zeros, which is what the gradient's last
// stage of a segment takes past its end: the padding is never read.
//
// Ten warps a CTA: warp 0 requests operands, warp 1 (even CTA) issues the MMAs,
// warps 2..9 store sums: two accumulators of 256 columns each let a tile's
// stores overlap the next one's MMAs.  Segments are found from the counts by
// every CTA, so a product is one launch and no list lives in memory.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>
#include <cstdint>

#include "gemm.h"
#include "grouped.h"
#include "kernels.h"
#include "pdl.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kMaxExperts = 256;
constexpr int kBK = 64;                              // K per stage: one 128-byte swizzle row
constexpr uint32_t kBoxBytes = 64 * 64 * 2;          // 64 x 64 bf16
constexpr int kTile = 256;                           // features and rows of a pair's tile
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;
constexpr int kStages = 6;
constexpr uint32_t kOperandBytes = 2 * kBoxBytes;    // a CTA's 128 rows of one operand
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kRowBox = 16;                          // rows of a box of a ragged tile
constexpr uint32_t kSmemBytes = kStages * kStageBytes + 256 + 1024;

enum Mode { kGemm, kGemmTransposed, kWgrad };

struct Maps {
  CUtensorMap a;        // product: W_e [experts][K][F] or [experts][F][K]; gradient: x
  CUtensorMap a_rows;   // gradient: x, one row a box (gather4)
  CUtensorMap b;        // rows of x / dy, full boxes
  CUtensorMap b_small;  // product: boxes of kRowBox rows
  CUtensorMap b_rows;   // one row a box (gather4)
};

struct Args {
  GroupArgs g;
  int gather_a, gather_b;
  uint32_t div_mul;     // id / slots
  int div_sh1, div_sh2;
  const float* add;
  void* out;
  int fp32;
  int na, nb;           // 256-wide tiles of the output: product: 1, features; gradient: columns of x, of dy
  int pairs;            // CTA pairs of the grid
};

struct Segments {
  int start[kMaxExperts], count[kMaxExperts], first[kMaxExperts + 1];   // first: row tiles before the expert's
  int ok;
};

// Segment starts and row tiles from the experts' counts (warp 0).  ok: the
// counts fit into max_rows rows.
__device__ __forceinline__ void find_segments(const GroupArgs& a, int lane, Segments& s) {
  long long row = 0;
  int tile = 0, bad = 0;
  for (int e0 = 0; e0 < a.N; e0 += 32) {
    const int e = e0 + lane;
    const int c = e < a.N ? a.counts[e] : 0;
    bad |= c < 0 || c > a.max_rows;
    const long long padded = bad ? 0 : ((long long)c + a.B - 1) / a.B * a.B;
    const int tiles = bad ? 0 : (c + kTile - 1) / kTile;
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
  bad = __any_sync(0xffffffffu, bad || row > a.max_rows);
  if (lane == 0) {
    s.first[a.N] = bad ? 0 : tile;
    s.ok = !bad;
    if (bad) atomicOr(a.status, kDevErrBadBlocks);
  }
}

// A tile of the output: product: rows row0 .. row0 + rows of the grouped
// tensors, features b; gradient: rows of the segment, columns a of x, b of dy.
struct Item {
  int e, row0, rows, a, b;
};

// Product: the items of an expert are contiguous and run in groups of G
// feature tiles x all of its row tiles, so that what runs at once shares its
// weight and row tiles through L2.  Gradient: the tiles of an expert, columns of
// dy fastest.  The order changes no bit of a tile.
template <Mode kMode>
__device__ __forceinline__ Item item_of(const Args& a, const Segments& s, int item) {
  Item it;
  if (kMode == kWgrad) {
    const int per = a.na * a.nb;
    it.e = item / per;
    const int l = item - it.e * per;
    it.a = l / a.nb;
    it.b = l - it.a * a.nb;
    it.row0 = s.start[it.e];
    it.rows = s.count[it.e];
  } else {
    const int t = item / a.nb;
    int lo = 0, hi = a.g.N;   // first[lo] <= t < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s.first[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const int first = s.first[lo], count = s.first[lo + 1] - first;
    const int l = item - first * a.nb;
    const int G = max(1, min(a.nb, (a.pairs + count - 1) / count));
    const int grp = l / (count * G), gsz = min(G, a.nb - grp * G), lin = l - grp * count * G;
    const int tile = lin / gsz;
    it.e = lo;
    it.a = 0;
    it.b = grp * G + lin - tile * gsz;
    it.row0 = s.start[lo] + tile * kTile;
    it.rows = min(kTile, s.count[lo] - tile * kTile);
  }
  return it;
}

// Rows of the tile that one CTA of the pair loads (half of the MMA's N).
__device__ __forceinline__ int half_rows(int rows) { return (rows + 31) / 32 * 16; }

// The row of a gathered operand that route r names, -1 (zeros) for none.
__device__ __forceinline__ int token_of(const Args& a, int r) {
  if ((uint32_t)r >= (uint32_t)(a.g.T * a.g.slots)) return -1;
  const uint32_t n = (uint32_t)r, t = __umulhi(a.div_mul, n);
  return (int)((t + ((n - t) >> a.div_sh1)) >> a.div_sh2);
}

// Rows p .. p + 3 of a gathered (or, with ids not wanted, in-place) operand;
// rows from `end` on are none.  p is a multiple of 4.
__device__ __forceinline__ int4 rows_of(const Args& a, bool gather, int p, int end) {
  int4 r = make_int4(-1, -1, -1, -1);
  if (p >= end) return r;
  if (gather) {
    const int4 id = __ldg(reinterpret_cast<const int4*>(a.g.ids + p));
    r = make_int4(token_of(a, id.x), token_of(a, id.y), token_of(a, id.z), token_of(a, id.w));
  } else {
    r = make_int4(p, p + 1, p + 2, p + 3);
  }
  if (p + 1 >= end) r.y = -1;
  if (p + 2 >= end) r.z = -1;
  if (p + 3 >= end) r.w = -1;
  return r;
}

__device__ __forceinline__ void store_bf16x8(uint16_t* p, const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

template <Mode kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    grouped_kernel(const __grid_constant__ Maps maps, const Args args) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Segments seg;
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  __shared__ int s_issued;            // stages the producer asked for
  __shared__ uint32_t s_tx[kStages];  // bytes of this CTA's last load into each stage
  __shared__ volatile PairEnd s_peer;

  const uint32_t rank = cluster_ctarank();   // 0: issues the MMAs
  const bool lead = rank == 0;
  const int pair0 = (int)(blockIdx.x >> 1), pairs = args.pairs;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * kStages;
  const uint32_t tfull0 = empty0 + 8 * kStages;
  const uint32_t tempty0 = tfull0 + 16;
  const uint32_t drain = tempty0 + 16;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wlim = args.g.wait_ns ? args.g.wait_ns : kWaitLimitNs;

  if (threadIdx.x == 32) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(full0 + 8 * st, 1);
      mbar_init(empty0 + 8 * st, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8 * b, 1);
      mbar_init(tempty0 + 8 * b, 2 * kEpiWarps);   // one arrival per epilogue warp of each CTA
    }
    mbar_init(drain, 1);
    s_abort = 0;
    s_peer.gave_up = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc_pair(smem_u32(&s_tmem_base), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&maps.a);
      prefetch_tmap(&maps.b);
      prefetch_tmap(&maps.b_small);
      prefetch_tmap(&maps.b_rows);
    }
    __syncwarp();
    // The set-up reads nothing an earlier kernel writes: it overlaps the end
    // of that kernel.  Earlier kernels' outputs are visible from here on.
    pdl_wait();
    find_segments(args.g, lane, seg);
  } else {
    pdl_wait();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  // every CTA of this persistent grid is resident: the next kernel may launch
  // now (it waits for this grid to finish)
  pdl_trigger();
  const uint32_t tmem = s_tmem_base;
  const int total = !seg.ok ? 0 : kMode == kWgrad ? args.g.N * args.na * args.nb : seg.first[args.g.N] * args.nb;
  const int ksteps_fixed = (args.g.K + kBK - 1) / kBK;
  auto ksteps_of = [&](const Item& it) { return kMode == kWgrad ? (it.rows + kBK - 1) / kBK : ksteps_fixed; };

  if (warp == 0) {
    // ------------------------------------------------------------ producer (both CTAs)
    const uint64_t pol_w = policy_evict_normal();
    const uint64_t pol_x = policy_evict_last();
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int item = pair0; item < total && ok; item += pairs) {
      const Item it = item_of<kMode>(args, seg, item);
      const int ksteps = ksteps_of(it), end = it.row0 + it.rows;
      // product: this CTA's rows of the tile; gradient: this CTA's columns
      const int half = half_rows(it.rows);
      const int brow0 = it.row0 + (int)rank * half;
      const int acol = it.a * kTile + (int)rank * 128, bcol = it.b * kTile + (int)rank * 128;
      int4 rows = {}, arows = {}, next = {}, anext = {};
      if (kMode != kWgrad) {
        if (args.gather_b && lane * 4 < half) rows = rows_of(args, true, brow0 + lane * 4, end);
      } else {
        const int p = it.row0 + (lane & 15) * 4;
        if (args.gather_a) anext = rows_of(args, true, p, end);
        if (args.gather_b) next = rows_of(args, true, p, end);
      }
      const uint32_t tx = kMode == kWgrad ? kStageBytes : kOperandBytes + (uint32_t)half * kBK * 2;
      for (int ks = 0; ks < ksteps; ++ks) {
        int got = 1;
        if (lane == 0) got = mbar_wait_cluster(empty0 + 8 * stage, phase ^ 1u, &s_abort, wlim) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          ok = false;
          break;
        }
        const uint32_t sA = smem_u32(smem + stage * kStageBytes), sB = sA + kOperandBytes;
        const uint32_t fb = mapa_shared(full0 + 8 * stage, 0);   // the even CTA's full barrier
        const int k0 = ks * kBK;
        if (lane == 0) {
          s_tx[stage] = tx;
          if (lead) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * tx);
        }
        if (kMode != kWgrad) {
          if (lane == 0) {
            if (kMode == kGemm) {
              tma_load_3d_pair(sA, &maps.a, bcol, k0, it.e, fb, pol_w);
              tma_load_3d_pair(sA + kBoxBytes, &maps.a, bcol + 64, k0, it.e, fb, pol_w);
            } else {
              tma_load_3d_pair(sA, &maps.a, k0, bcol, it.e, fb, pol_w);
            }
          }
          if (args.gather_b) {
            if (lane * 4 < half) tma_gather4_pair(sB + lane * 512, &maps.b_rows, k0, rows, fb, pol_x);
          } else if (half == 128) {
            if (lane == 0) tma_load_2d_pair(sB, &maps.b, k0, brow0, fb, pol_x);
          } else if (lane * kRowBox < half) {
            tma_load_2d_pair(sB + lane * kRowBox * 128, &maps.b_small, k0, brow0 + lane * kRowBox, fb, pol_x);
          }
        } else {
          // the segment's last rows, too, one row at a time: rows past its end
          // are none and read zeros
          const int p0 = it.row0 + k0, p = p0 + (lane & 15) * 4;
          const bool tail = p0 + kBK > end;
          arows = args.gather_a ? anext : rows_of(args, false, p, end);
          rows = args.gather_b ? next : rows_of(args, false, p, end);
          const uint32_t at = (uint32_t)(lane >> 4) * kBoxBytes + (uint32_t)(lane & 15) * 512;
          const int box = (lane >> 4) * 64;
          if (args.gather_a || tail)
            tma_gather4_pair(sA + at, &maps.a_rows, acol + box, arows, fb, pol_x);
          else if (lane < 2)
            tma_load_2d_pair(sA + lane * kBoxBytes, &maps.a, acol + lane * 64, p0, fb, pol_x);
          if (args.gather_b || tail)
            tma_gather4_pair(sB + at, &maps.b_rows, bcol + box, rows, fb, pol_x);
          else if (lane < 2)
            tma_load_2d_pair(sB + lane * kBoxBytes, &maps.b, bcol + lane * 64, p0, fb, pol_x);
          // the next stage's routes, asked for a stage ahead
          if (args.gather_a) anext = rows_of(args, true, p + kBK, end);
          if (args.gather_b) next = rows_of(args, true, p + kBK, end);
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      s_abort = 1;
      if (lane == 0) atomicOr(args.g.status, kDevErrTimeout);
    }
    if (lane == 0) s_issued = issued;
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lead && lane == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      // descriptors of stage 0, K step 0; a K = 16 step adds 2 KB to an
      // MN-major operand (64-wide atoms 8 KB apart, 8-row K groups 1 KB) and
      // 32 B to a K-major one, in the 16-byte units of the address field
      constexpr bool kAMn = kMode != kGemmTransposed, kBMn = kMode == kWgrad;
      constexpr uint32_t kAStep = kAMn ? 128 : 2, kBStep = kBMn ? 128 : 2;
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), kAMn ? kBoxBytes : 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(smem) + kOperandBytes, kBMn ? kBoxBytes : 16, 1024);
      uint32_t soff = 0;
      for (int item = pair0; item < total && ok; item += pairs) {
        const Item it = item_of<kMode>(args, seg, item);
        const int ksteps = ksteps_of(it);
        if (ksteps == 0) continue;   // an expert without rows: nothing to sum
        const uint32_t idesc = idesc_bf16(kTile, kMode == kWgrad ? kTile : 2 * half_rows(it.rows), kAMn, kBMn);
        if (!mbar_wait_cluster(tempty0 + 8 * acc, acc_phase ^ 1u, &s_abort, wlim)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d0 = tmem + acc * kTile;
        for (int ks = 0; ks < ksteps; ++ks) {
          if (!mbar_wait_cluster(full0 + 8 * stage, phase, &s_abort, wlim)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = adesc0 + soff, bd = bdesc0 + soff;
          const int left = (kMode == kWgrad ? it.rows : args.g.K) - ks * kBK;   // K left: zeros from there on
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            if (kk * 16 < left) mma_bf16_pair(d0, ad + kk * kAStep, bd + kk * kBStep, idesc, (ks | kk) != 0 ? 1u : 0u);
          mma_commit_pair(empty0 + 8 * stage, 0x3);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
            soff = 0;
          } else {
            soff += kStageBytes >> 4;
          }
        }
        if (!ok) break;
        mma_commit_pair(tfull0 + 8 * acc, 0x3);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok) {
        s_abort = 1;
        atomicOr(args.g.status, kDevErrTimeout);
      }
      // all issued MMAs must be complete before TMEM is released
      mma_commit_pair(drain, 0x3);
      volatile int no_abort = 0;
      mbar_wait(drain, 0, &no_abort);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3;                       // TMEM lanes this warp may access
    const int col0 = ((warp - 2) / 4) * (kTile / 2);    // its half of the 256 columns
    const int F = args.g.F;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int item = pair0; item < total; item += pairs) {
      const Item it = item_of<kMode>(args, seg, item);
      const bool empty = kMode == kWgrad && it.rows == 0;
      if (!empty) {
        int got = 1;
        if (lane == 0) got = mbar_wait_cluster(tfull0 + 8 * acc, acc_phase, &s_abort, wlim) ? 1 : 0;
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          if (lane == 0) {
            s_abort = 1;
            atomicOr(args.g.status, kDevErrTimeout);
          }
          break;
        }
        tc_fence_after();
      }
      const uint32_t tbase = tmem + ((uint32_t)(quarter * 32) << 16) + acc * kTile;
      if (kMode != kWgrad) {
        // a lane is an output feature, a column a row of y
        const int feat = it.b * kTile + (int)rank * 128 + quarter * 32 + lane;
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(args.out) + (size_t)it.row0 * F + feat;
        for (int c = col0; c < col0 + kTile / 2 && c < it.rows; c += 16) {
          float v[16];
          tmem_ld16(tbase + c, v);
          tmem_wait_ld();
          if (feat < F) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < it.rows) out[(size_t)(c + j) * F] = __float2bfloat16_rn(v[j]);
          }
          __syncwarp();   // tmem_ld16 is one instruction of the whole warp
        }
      } else {
        // a lane is a column of x, a column one of dy: contiguous in dw
        const int m = it.a * kTile + (int)rank * 128 + quarter * 32 + lane;
        const size_t row = ((size_t)it.e * args.g.K + m) * F;
        for (int c = col0; c < col0 + kTile / 2; c += 16) {
          const int n = it.b * kTile + c;
          if (n >= F) break;   // the same for the whole warp
          float v[16];
          if (!empty) {
            tmem_ld16(tbase + c, v);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.0f;
          }
          if (m < args.g.K) {
#pragma unroll
            for (int h = 0; h < 16; h += 8) {
              if (n + h >= F) break;
              if (!args.fp32) {
                store_bf16x8(reinterpret_cast<uint16_t*>(args.out) + row + n + h, v + h);
              } else {
                float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(args.out) + row + n + h);
                float4 q[2] = {make_float4(v[h], v[h + 1], v[h + 2], v[h + 3]),
                               make_float4(v[h + 4], v[h + 5], v[h + 6], v[h + 7])};
                if (args.add) {   // add may be out (no __restrict__): read before it is written
                  const float4* d = reinterpret_cast<const float4*>(args.add + row + n + h);
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    const float4 z = __ldcs(d + i);
                    q[i] = make_float4(z.x + q[i].x, z.y + q[i].y, z.z + q[i].z, z.w + q[i].w);
                  }
                }
                __stcs(o, q[0]);
                __stcs(o + 1, q[1]);
              }
            }
          }
          __syncwarp();
        }
      }
      if (empty) continue;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_shared(tempty0 + 8 * acc, 0));
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  end_pair(lead, full0, drain, kStages, s_issued, s_abort, &s_peer, [&](int i) {
    // a load that only the other CTA asked for: a pair's loads have the same size
    return s_tx[i % kStages];
  });
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------ host
bool encode(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* m, const void* base, int rank, uint64_t d0, uint64_t d1,
            uint64_t d2, uint32_t b0, uint32_t b1) {
  const cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {2 * d0, 2 * d0 * d1};
  const cuuint32_t box[3] = {b0, b1, 1}, estr[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// id / d = (t + ((id - t) >> sh1)) >> sh2, t = the upper half of mul * id
// (division by an invariant, Granlund and Montgomery 1994)
void set_divisor(Args& a, uint32_t d) {
  int l = 0;
  while ((1ull << l) < d) ++l;
  a.div_mul = (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
  a.div_sh1 = l < 1 ? l : 1;
  a.div_sh2 = l < 1 ? 0 : l - 1;
}

// Pairs of CTAs that can be resident at once, looked up once per device and kernel.
template <Mode kMode>
int resident_pairs(int sms) {
  static int cache[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
  cudaFuncSetAttribute(grouped_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)(sms / 2), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, grouped_kernel<kMode>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = sms / 2;
  }
  n = n < sms / 2 ? n : sms / 2;
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

template <Mode kMode>
void launch(const Maps& m, Args& a, long long items, int sms, cudaStream_t s) {
  const int cap = resident_pairs<kMode>(sms);
  a.pairs = (int)(items < cap ? items : cap);
  launch_pdl(grouped_kernel<kMode>, dim3(2 * a.pairs), dim3(kThreads), kSmemBytes, s, m, a);
}

// The rows that experts hold in all, at most.
long long routes_of(const GroupArgs& g) {
  const long long r = (long long)g.T * g.slots;
  return r < g.max_rows ? r : g.max_rows;
}

}  // namespace

bool launch_grouped_gemm(const GroupedGemmArgs& in, PFN_cuTensorMapEncodeTiled_v12000 fn, int sms, cudaStream_t s) {
  const GroupArgs& g = in.g;
  const uint64_t K = g.K, F = g.F, N = g.N, rows = in.gather ? (uint64_t)g.T : (uint64_t)g.max_rows;
  Maps m{};
  if (!(in.transposed ? encode(fn, &m.a, in.w, 3, K, F, N, kBK, 128) : encode(fn, &m.a, in.w, 3, F, K, N, 64, kBK)) ||
      !encode(fn, &m.b, in.x, 2, K, rows, 1, kBK, 128) || !encode(fn, &m.b_small, in.x, 2, K, rows, 1, kBK, kRowBox) ||
      !encode(fn, &m.b_rows, in.x, 2, K, rows, 1, kBK, 1))
    return false;
  m.a_rows = m.b_rows;
  Args a{};
  a.g = g;
  a.gather_b = in.gather;
  set_divisor(a, (uint32_t)g.slots);
  a.out = in.y;
  a.na = 1;
  a.nb = (g.F + kTile - 1) / kTile;
  const long long routes = routes_of(g), tiles = routes / kTile + (routes < g.N ? routes : g.N);
  if (in.transposed)
    launch<kGemmTransposed>(m, a, tiles * a.nb, sms, s);
  else
    launch<kGemm>(m, a, tiles * a.nb, sms, s);
  return true;
}

bool launch_grouped_wgrad(const GroupedWgradArgs& in, PFN_cuTensorMapEncodeTiled_v12000 fn, int sms, cudaStream_t s) {
  const GroupArgs& g = in.g;
  const uint64_t K = g.K, F = g.F, xr = in.gather_x ? (uint64_t)g.T : (uint64_t)g.max_rows,
                 dr = in.gather_dy ? (uint64_t)g.T : (uint64_t)g.max_rows;
  Maps m{};
  if (!encode(fn, &m.a, in.x, 2, K, xr, 1, 64, kBK) || !encode(fn, &m.a_rows, in.x, 2, K, xr, 1, 64, 1) ||
      !encode(fn, &m.b, in.dy, 2, F, dr, 1, 64, kBK) || !encode(fn, &m.b_rows, in.dy, 2, F, dr, 1, 64, 1))
    return false;
  m.b_small = m.b_rows;
  Args a{};
  a.g = g;
  a.gather_a = in.gather_x;
  a.gather_b = in.gather_dy;
  set_divisor(a, (uint32_t)g.slots);
  a.add = in.add;
  a.out = in.dw;
  a.fp32 = in.fp32;
  a.na = (g.K + kTile - 1) / kTile;
  a.nb = (g.F + kTile - 1) / kTile;
  launch<kWgrad>(m, a, (long long)g.N * a.na * a.nb, sms, s);
  return true;
}

}  // namespace moe
