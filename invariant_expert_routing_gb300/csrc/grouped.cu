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
//             transpose, features of K: K-major), twice for items of two groups
//             (wide_items), B = up to 256 rows of x (K-major).  The MMA's N is
//             the tile's rows rounded up to 32: columns of an MMA are
//             independent sums over the same K steps, so a row's bits depend
//             neither on N nor on the batch.  An expert's tiles are of one
//             height, to 32 rows: full ones and a short last one took 297 us
//             for 281 (W13 of 8192 tokens in the 128-expert layer), 608 for 570
//             (W2's input gradient in the 8-expert layer).
//   gradient: A = 256 columns of x, B = 256 columns of dy, both MN-major, K
//             the expert's rows in ascending order.
// Rows gathered by route come by TMA gather4, four rows a request, straight from
// the token tensor: no copy in segment order.  A row index outside the tensor
// reads zeros, which is what the gradient's last rows of a segment ask for past
// its end: the padding is never read.
//
// Warps 0 and 10..14 request operands (10..14 in launches that may gather: they
// take the stages in turn), warp 1 (even CTA) issues the MMAs, warps 2..9 store
// sums.  The requesting and issuing warps run converged and elect a lane for a
// stage's requests, all in one block: descriptors and coordinates stay in
// uniform registers, and a warp that came together after each request took 300
// cycles more for it (the MMAs of a stage take 512; a loop of one lane took 85
// for a request).  Two accumulators of 256 columns each let a tile's stores
// overlap the next one's MMAs.  Segments are found from the counts by every CTA,
// so a product is one launch and no list lives in memory.
//
// Times here are of one of the first 50 calls unless they are called sustained: a
// loop of large products runs into the power cap, which takes the clock from 2070 to
// some 1400 to 1700 MHz and a call up to 15 % longer.
//
// Bounds.  Two experts of about 4096 rows, 4096 x 14336 in place: 1840 TFLOP/s of the
// measured 1916 the product, 1600 the bf16 gradient.  Sustained, in cycles of the
// clock that was seen, the tensor pipe is busy 85 % in the 8-expert layer's input
// gradient of W2 (4096 tokens) in place and 76 % gathered (658 and 670 us): the
// requests of gathered rows, some 16 cycles a gather4 and 32 of them a stage, are the
// difference.  In the 128-expert layer's W13 (8192 tokens) it is 67 % in place and
// 62 % gathered (327 and 328 us): items of unequal height are handed out by number,
// a two-group item's stores overlap no MMAs, and rows are rounded up to 32.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>
#include <cmath>
#include <cstdint>

#include "gemm.h"
#include "grouped.h"
#include "kernels.h"
#include "mx.cuh"
#include "pdl.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kMaxExperts = 256;
constexpr int kBK = 64;                              // K per stage: one 128-byte swizzle row
constexpr uint32_t kBoxBytes = 64 * 64 * 2;          // 64 x 64 bf16
constexpr int kTile = 256;                           // features and rows of a pair's tile
constexpr int kEpiWarps = 8;
constexpr int kThreads = (2 + kEpiWarps) * 32;       // with one requesting warp
constexpr uint32_t kOperandBytes = 2 * kBoxBytes;    // a CTA's 128 rows of one operand
constexpr int kRowBox = 16;                          // rows of a box of a ragged tile
constexpr uint32_t kRowBoxBytes = kRowBox * 128 * 2;   // of an MN-major operand: 128 columns

enum Mode { kGemm, kGemmWide, kGemmTransposed, kGemmTransposedWide, kWgrad, kWgradAdd };
__host__ __device__ constexpr bool transposed(Mode m) { return m == kGemmTransposed || m == kGemmTransposedWide; }
__host__ __device__ constexpr int groups(Mode m) { return m == kGemmWide || m == kGemmTransposedWide ? 2 : 1; }
__host__ __device__ constexpr bool wgrad(Mode m) { return m >= kWgrad; }

// A gradient sums at most this many stages of 64 rows in an accumulator.  The
// tensor cores truncate each 16-row step's sum to fp32: 1e-6 of the result for
// 1024 rows, 1e-5 for 8192 (2-norms; rounded sums would stay at 3e-7).  Longer
// segments are summed part by part, the parts added (rounded to nearest) in the
// other accumulator's columns, and the MMAs wait for that.  For bf16 results 1e-5
// is nothing, and products, always bf16, are summed in one part whatever K: with K
// 2048 and 4096 one result in 850 and in 420 rounds to the other neighbour than a
// sum rounded at every step, and the error against 64 bits (1.66e-3 in the 2-norm,
// the rounding to bf16) is the same in six digits.
constexpr int kPartStagesFp32 = 12, kPartStagesBf16 = 128;

// kWgradAdd reads and writes fp32 gradients at the rate of memory: four stages
// keep its MMAs fed, and 64 KB hold what the next sums are added to (two blocks
// of 32 rows x 128 bytes an epilogue warp; 32 registers a lane instead, half as
// much in flight: 730 us for 8192 tokens in the 128-expert layer).
constexpr uint32_t kAddBlock = 32 * 128;
template <Mode kMode>
struct Cfg {
  static constexpr int kGroups = groups(kMode);   // 256-feature groups of an item
  static constexpr uint32_t kABytes = kGroups * kOperandBytes, kStageBytes = kABytes + kOperandBytes;
  static constexpr int kStages = kMode == kWgradAdd || kGroups > 1 ? 4 : 6;
  // Requesting warps of a launch that may gather.  A warp that asked for stage
  // number n goes on to n + kParts knowing that n - kStages was consumed; for the
  // parity of the stage's barrier to tell its phases apart, n + kParts - 2 kStages
  // has to be.
  static constexpr int kParts = kStages;
  static_assert(kParts <= kStages, "a requesting warp could overwrite a stage in use");
  static constexpr int kMaxThreads = kThreads + (kParts - 1) * 32;
  static constexpr uint32_t kAddBytes = kMode == kWgradAdd ? kEpiWarps * 2 * kAddBlock : 0;
  static constexpr uint32_t kSmemBytes = kStages * kStageBytes + kAddBytes + 256 + 1024;
};

struct Maps {
  CUtensorMap a;        // product: W_e [experts][K][F] or [experts][F][K]; gradient: x
  CUtensorMap b;        // gradient: dy, full boxes
  CUtensorMap b_box[4];   // product: x, 16, 32, 64 and 128 rows a box
  CUtensorMap a_small, b_small;   // gradient: kRowBox rows a box
  CUtensorMap a_rows, b_rows;     // one row a box: gather4 (a: gradient)
};

struct Args {
  GroupArgs g;
  int gather_a, gather_b;
  int wide_a, wide_b;   // MN-major operands whose 128 features are one box (two otherwise)
  uint32_t div_mul;     // id / slots
  int div_sh1, div_sh2;
  const float* add;
  void* out;
  int fp32;
  int wide_out;         // out takes 32-byte stores
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
  if (wgrad(kMode)) {
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
    const int rows = ((s.count[lo] + count - 1) / count + 31) & ~31;   // (at most 256; the last tile has some)
    it.row0 = s.start[lo] + tile * rows;
    it.rows = min(rows, s.count[lo] - tile * rows);
  }
  it.e = mx::uniform(it.e);
  it.row0 = mx::uniform(it.row0);
  it.rows = mx::uniform(it.rows);
  it.a = mx::uniform(it.a);
  it.b = mx::uniform(it.b);
  return it;
}

// A wait of a converged warp: every lane sees the barrier, and they agree.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, limit));
}
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit) {
  return __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, abort, limit));
}

// Rows of the tile that one CTA of the pair loads (half of the MMA's N).
__device__ __forceinline__ int half_rows(int rows) { return (rows + 31) / 32 * 16; }

// The row of a gathered operand that route r names, -1 (zeros) for none.
__device__ __forceinline__ int token_of(const Args& a, int r) {
  if ((uint32_t)r >= (uint32_t)(a.g.T * a.g.slots)) return -1;
  const uint32_t n = (uint32_t)r, t = __umulhi(a.div_mul, n);
  return (int)((t + ((n - t) >> a.div_sh1)) >> a.div_sh2);
}

// Four rows for a gather4, p on; p is a multiple of 4 (a segment's start is one of 8).
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

// One operand of a gradient's stage: 64 rows p0 on, 128 columns col on.  The
// whole box if 64 rows in place are left; otherwise 16 rows at a time, by box if
// they are in place and all there, by gather4 if not (rows: the 64 rows).
struct Operand {
  const CUtensorMap *box, *small, *rows;
  bool gather, wide;
};
__device__ __forceinline__ uint32_t operand_bytes(bool gather, int left) {
  return !gather && left >= kBK ? kOperandBytes : (uint32_t)min(kBK / kRowBox, (left + kRowBox - 1) / kRowBox) * kRowBoxBytes;
}
__device__ __forceinline__ void request_operand(const Operand& o, uint32_t dst, int col, int p0, int left, const int4* rows,
                                                uint32_t bar, uint64_t policy) {
  if (!o.gather && left >= kBK) {
    if (o.wide) {
      mx::tma_load_3d_pair(dst, o.box, 0, p0, col >> 6, bar, policy);
    } else {
      tma_load_2d_pair(dst, o.box, col, p0, bar, policy);
      tma_load_2d_pair(dst + kBoxBytes, o.box, col + 64, p0, bar, policy);
    }
    return;
  }
  for (int r0 = 0; r0 < min(left, kBK); r0 += kRowBox) {
    const uint32_t at = dst + r0 * 128;
    if (!o.gather && r0 + kRowBox <= left) {
      // (one box of 128 columns would put its halves 2 KB apart)
      tma_load_2d_pair(at, o.small, col, p0 + r0, bar, policy);
      tma_load_2d_pair(at + kBoxBytes, o.small, col + 64, p0 + r0, bar, policy);
      continue;
    }
#pragma unroll
    for (int i = 0; i < kRowBox / 4; ++i) {
      const int4 r = rows[r0 / 4 + i];
      tma_gather4_pair(at + i * 512, o.rows, col, r.x, r.y, r.z, r.w, bar, policy);
      tma_gather4_pair(at + i * 512 + kBoxBytes, o.rows, col + 64, r.x, r.y, r.z, r.w, bar, policy);
    }
  }
}

// How a CTA's requesting warps ended, told to the other CTA of the pair.
constexpr int kMostParts = 6;
struct PartsEnd {
  int issued[kMostParts], gave_up;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Among four lanes in turn, each with a row of four 32-byte blocks: lane q's
// block j becomes lane j's block q, so that four lanes hold 128 bytes of a row
// (an access of 32 bytes a row is a request of its own to L2: 454 us for the
// fp32 gradients of 8192 tokens in the 128-expert layer).
__device__ __forceinline__ void transpose4(float (&v)[32], int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (b & bit) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float &lo = v[8 * b + i], &hi = v[8 * (b | bit) + i];
        const float got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
        if (up)
          lo = got;
        else
          hi = got;
      }
    }
  }
}

// 32 bytes: one access where the address is 32-byte aligned (a whole sector), two
// otherwise.
__device__ __forceinline__ void store8(void* p, bool wide, const uint32_t* w) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(reinterpret_cast<uint4*>(p) + 1, make_uint4(w[4], w[5], w[6], w[7]));
  }
}

template <Mode kMode>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<kMode>::kMaxThreads, 1)
    grouped_kernel(const __grid_constant__ Maps maps, const Args args) {
  constexpr int kStages = Cfg<kMode>::kStages, kParts = Cfg<kMode>::kParts, kGroups = Cfg<kMode>::kGroups;
  constexpr uint32_t kABytes = Cfg<kMode>::kABytes, kStageBytes = Cfg<kMode>::kStageBytes;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Segments seg;
  __shared__ uint32_t s_tmem_base;
  __shared__ volatile int s_abort;
  __shared__ PartsEnd s_end;          // stages that each requesting warp asked for
  __shared__ uint32_t s_tx[kStages];  // bytes of this CTA's last load into each stage
  __shared__ volatile PartsEnd s_peer;
  __shared__ int4 s_rows[kParts][32]; // rows of a requesting warp's gather4 requests

  const uint32_t rank = cluster_ctarank();   // 0: issues the MMAs
  const bool lead = rank == 0;
  const int pair0 = (int)(blockIdx.x >> 1), pairs = args.pairs;

  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* adds = smem + kStages * kStageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(adds + Cfg<kMode>::kAddBytes);
  const uint32_t full0 = smem_u32(bars);
  const uint32_t empty0 = full0 + 8 * kStages;
  const uint32_t tfull0 = empty0 + 8 * kStages;
  const uint32_t tempty0 = tfull0 + 16;
  const uint32_t drain = tempty0 + 16;
  const int parts = wgrad(kMode) || args.gather_b ? kParts : 1;   // requesting warps

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
    for (int w = 0; w < kParts; ++w) s_end.issued[w] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc_pair(smem_u32(&s_tmem_base), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(args.gather_a ? &maps.a_rows : &maps.a);
      prefetch_tmap(args.gather_b ? &maps.b_rows : wgrad(kMode) ? &maps.b : &maps.b_box[3]);
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
  const uint32_t tmem = (uint32_t)mx::uniform((int)s_tmem_base);
  const int total = mx::uniform(!seg.ok ? 0 : wgrad(kMode) ? args.g.N * args.na * args.nb : seg.first[args.g.N] * args.nb);
  const int ksteps_fixed = (args.g.K + kBK - 1) / kBK;
  auto ksteps_of = [&](const Item& it) { return wgrad(kMode) ? (it.rows + kBK - 1) / kBK : ksteps_fixed; };
  // Stages that go into one accumulator of a tile (all of them, or a part's).
  auto part_of = [&](int ksteps) {
    const int most = args.fp32 ? kPartStagesFp32 : kPartStagesBf16;
    return !wgrad(kMode) || ksteps <= most ? ksteps : most;
  };

  if (warp == 0 || warp >= 2 + kEpiWarps) {
    // ------------------------------------------------------------ producers (both CTAs)
    const int part = warp == 0 ? 0 : mx::uniform(warp - (1 + kEpiWarps));
    const uint64_t pol_w = policy_evict_normal();
    const uint64_t pol_x = policy_evict_last();
    const uint32_t s0 = smem_u32(smem);
    const int me = mx::uniform((int)rank);
    const uint32_t full_lead = mapa_shared(full0, 0);   // the even CTA's full barriers
    const Operand oa{&maps.a, &maps.a_small, &maps.a_rows, args.gather_a != 0, args.wide_a != 0};
    const Operand ob{&maps.b, &maps.b_small, &maps.b_rows, args.gather_b != 0, args.wide_b != 0};
    int4* rows = s_rows[part];
    int n0 = 0, issued = 0;   // stages of the items before; this warp's
    bool ok = true;
    for (int item = pair0; item < total && ok; item += pairs) {
      const Item it = item_of<kMode>(args, seg, item);
      const int ksteps = ksteps_of(it), end = it.row0 + it.rows;
      // product: this CTA's rows of the tile; gradient: this CTA's columns
      const int half = half_rows(it.rows);
      const int brow0 = it.row0 + me * half;
      // product in place: the largest box that fits, twice (the second one's last
      // row is the last) if it does not fill the rows (boxes of 16 rows instead: 357
      // us for 290, W13 of 8192 tokens in the 128-expert layer)
      const int box = 31 - __clz(max(half, 16)), box_rows = 1 << box, boxes = half == box_rows ? 1 : 2;
      const int acol = it.a * kTile + me * 128, bcol = it.b * kGroups * kTile + me * 128;
      const int first = (part + parts - n0 % parts) % parts;   // this warp's first stage of the item
      int4 next = {};   // gradient: rows of the next stage, x in lanes 0..15, dy in lanes 16..31
      const bool gather_mine = lane < 16 ? oa.gather : ob.gather;
      if (wgrad(kMode)) {
        next = rows_of(args, gather_mine, it.row0 + first * kBK + (lane & 15) * 4, end);
      } else if (args.gather_b) {
        __syncwarp();
        if (4 * lane < half) rows[lane] = rows_of(args, true, brow0 + 4 * lane, end);
        __syncwarp();
      }
      for (int ks = first; ks < ksteps; ks += parts) {
        const int p0 = it.row0 + ks * kBK, left = it.rows - ks * kBK;
        if (wgrad(kMode)) {
          // the stage's rows are in the table before the stage is free, the next one's asked for
          __syncwarp();
          rows[lane] = next;
          __syncwarp();
          next = rows_of(args, gather_mine, p0 + parts * kBK + (lane & 15) * 4, end);
        }
        const int n = n0 + ks, stage = n % kStages;
        const uint32_t phase = (uint32_t)(n / kStages) & 1u;
        if (!warp_wait(empty0 + 8 * stage, phase ^ 1u, &s_abort, wlim)) {
          ok = false;
          break;
        }
        const uint32_t sA = s0 + stage * kStageBytes, sB = sA + kABytes;
        const uint32_t fb = full_lead + 8 * stage;
        const int k0 = ks * kBK;
        if (!wgrad(kMode)) {
          if (mx::elect_one()) {
            const uint32_t tx = kABytes + (uint32_t)(args.gather_b ? half : boxes * box_rows) * kBK * 2;
            s_tx[stage] = tx;
            if (lead) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * tx);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
              const uint32_t to = sA + g * kOperandBytes;
              const int col = bcol + g * kTile;
              if (transposed(kMode)) {
                mx::tma_load_3d_pair(to, &maps.a, k0, col, it.e, fb, pol_w);
              } else if (args.wide_a) {
                tma_load_4d_pair(to, &maps.a, 0, k0, col >> 6, it.e, fb, pol_w);
              } else {
                mx::tma_load_3d_pair(to, &maps.a, col, k0, it.e, fb, pol_w);
                mx::tma_load_3d_pair(to + kBoxBytes, &maps.a, col + 64, k0, it.e, fb, pol_w);
              }
            }
            if (args.gather_b) {
#pragma unroll 8
              for (int i = 0; i < half / 4; ++i) {
                const int4 r = rows[i];
                tma_gather4_pair(sB + i * 512, &maps.b_rows, k0, r.x, r.y, r.z, r.w, fb, pol_x);
              }
            } else {
              const CUtensorMap* m = &maps.b_box[box - 4];
              tma_load_2d_pair(sB, m, k0, brow0, fb, pol_x);
              if (boxes == 2) tma_load_2d_pair(sB + (half - box_rows) * 128, m, k0, brow0 + half - box_rows, fb, pol_x);
            }
          }
        } else {
          if (mx::elect_one()) {
            const uint32_t tx = operand_bytes(oa.gather, left) + operand_bytes(ob.gather, left);
            s_tx[stage] = tx;
            if (lead) mbar_arrive_expect_tx(full0 + 8 * stage, 2 * tx);
            request_operand(oa, sA, acol, p0, left, rows, fb, pol_x);
            request_operand(ob, sB, bcol, p0, left, rows + 16, fb, pol_x);
          }
        }
        __syncwarp();
        ++issued;
      }
      n0 += ksteps;
    }
    if (!ok) {
      s_abort = 1;
      if (lane == 0) atomicOr(args.g.status, kDevErrTimeout);
    }
    if (lane == 0) s_end.issued[part] = issued;
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (lead) {
      const bool leader = mx::elect_one();
      int stage = 0, acc = 0;
      uint32_t phase = 0, taken = 0;   // taken: parity of each accumulator's uses
      bool ok = true;
      auto take = [&](int b) {         // the accumulator's sums have been read
        const bool got = warp_wait_cluster(tempty0 + 8 * b, ((taken >> b) & 1u) ^ 1u, &s_abort, wlim);
        taken ^= 1u << b;
        tc_fence_after();
        return got;
      };
      // descriptors of stage 0, K step 0; a K = 16 step adds 2 KB to an
      // MN-major operand (64-wide atoms 8 KB apart, 8-row K groups 1 KB) and
      // 32 B to a K-major one, in the 16-byte units of the address field
      constexpr bool kAMn = !transposed(kMode), kBMn = wgrad(kMode);
      constexpr uint32_t kAStep = kAMn ? 128 : 2, kBStep = kBMn ? 128 : 2;
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), kAMn ? kBoxBytes : 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(smem) + kABytes, kBMn ? kBoxBytes : 16, 1024);
      uint32_t soff = 0;
      for (int item = pair0; item < total && ok; item += pairs) {
        const Item it = item_of<kMode>(args, seg, item);
        const int ksteps = ksteps_of(it);
        if (ksteps == 0) continue;   // an expert without rows: nothing to sum
        const uint32_t idesc = idesc_bf16(kTile, wgrad(kMode) ? kTile : 2 * half_rows(it.rows), kAMn, kBMn);
        const int part_stages = part_of(ksteps);
        int left_in_part = 0;
        const uint32_t d0 = tmem + acc * kTile;
        for (int ks = 0; ok && ks < ksteps; ++ks) {
          const bool first = left_in_part == 0;
          if (first) {
            left_in_part = min(part_stages, ksteps - ks);
            ok = take(acc);
            if (!ok) break;
          }
          --left_in_part;
          if (!warp_wait_cluster(full0 + 8 * stage, phase, &s_abort, wlim)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t ad = adesc0 + soff, bd = bdesc0 + soff;
          const int left = (wgrad(kMode) ? it.rows : args.g.K) - ks * kBK;   // K left: zeros from there on
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
              if (kk * 16 < left) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g)
                  mma_bf16_pair(d0 + g * kTile, ad + g * (kOperandBytes >> 4) + kk * kAStep, bd + kk * kBStep, idesc,
                                !first || kk != 0 ? 1u : 0u);
              }
            mma_commit_pair(empty0 + 8 * stage, 0x3);
            if (left_in_part == 0) mma_commit_pair(tfull0 + 8 * acc, 0x3);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
            soff = 0;
          } else {
            soff += kStageBytes >> 4;
          }
        }
        if (!ok) break;
        // A segment in parts is added up in the other accumulator, which the epilogue
        // warps had read before they came to it: it counts as taken once all its parts
        // have been issued (all warps are past the first then), and the next item
        // starts in this one while they store from that one.
        if (ksteps > part_stages)
          ok = take(acc ^ 1);
        else if (kGroups == 1)
          acc ^= 1;
      }
      if (!ok) {
        s_abort = 1;
        if (lane == 0) atomicOr(args.g.status, kDevErrTimeout);
      }
      // all issued MMAs must be complete before TMEM is released
      if (leader) mma_commit_pair(drain, 0x3);
      __syncwarp();
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
    uint32_t seen = 0;   // parity of each accumulator's full phases
    auto wait_full = [&]() {
      int got = 1;
      if (lane == 0) got = mbar_wait_cluster(tfull0 + 8 * acc, (seen >> acc) & 1u, &s_abort, wlim) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      seen ^= 1u << acc;
      if (!got && lane == 0) {
        s_abort = 1;
        atomicOr(args.g.status, kDevErrTimeout);
      }
      tc_fence_after();
      return got != 0;
    };
    auto release = [&](int b) {   // this warp has read what it needs of accumulator b
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mx::mbar_arrive_remote_relaxed(mapa_shared(tempty0 + 8 * b, 0));
    };
    // Gradient: this warp's blocks of 32 columns of a tile that lie in dw (the
    // first ones; none if its rows do not).
    auto blocks_of = [&](const Item& of) {
      const int m = of.a * kTile + (int)rank * 128 + quarter * 32, n = F - of.b * kTile - col0;
      return m >= args.g.K || n <= 0 ? 0 : min(4, (n + 31) / 32);
    };
    // kWgradAdd: what the sums are added to comes two blocks (of 32 columns) ahead,
    // the first two of an item during the one before.  Whole lines are requested, 8
    // lanes a row; the chunks of a row's 128 bytes are swapped in pairs by bit 2 of
    // the row, so that the lanes that read a block meet different banks.
    const uint32_t add0 = smem_u32(adds) + (uint32_t)(warp - 2) * 2 * kAddBlock;
    auto request_add = [&](const Item& of, int block) {
      const int n = of.b * kTile + col0 + block * 32 + (lane & 7) * 4;
      const int m = of.a * kTile + (int)rank * 128 + quarter * 32;
      if (block < blocks_of(of)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3);
          const bool in = m + r < args.g.K && n < F;
          const float* src = in ? args.add + ((size_t)of.e * args.g.K + m + r) * F + n : args.add;
          cp_async16(add0 + (block & 1) * kAddBlock + r * 128 + (((lane & 7) ^ (i & 1)) << 4), src, in ? 16 : 0);
        }
      }
      cp_async_commit();
    };
    if (kMode == kWgradAdd && pair0 < total) {
      const Item it = item_of<kMode>(args, seg, pair0);
      request_add(it, 0);
      request_add(it, 1);
    }
    for (int item = pair0; item < total; item += pairs) {
      const Item it = item_of<kMode>(args, seg, item);
      const bool empty = wgrad(kMode) && it.rows == 0;
      // Gradient: TMEM lanes are columns of x, its columns those of dy, contiguous
      // in dw.  After transpose4 a lane has 32 bytes (block lane & 3 of 128) of rows
      // m0 .. m0 + 3.
      const int per = args.fp32 ? 8 : 16;   // elements of a block
      const int m0 = it.a * kTile + (int)rank * 128 + quarter * 32 + (lane & ~3);
      const int n0 = it.b * kTile + col0, nl = n0 + (lane & 3) * per;
      const size_t at = ((size_t)it.e * args.g.K + m0) * F + nl;
      const bool wide = args.wide_out != 0;
      const uint32_t tlane = tmem + ((uint32_t)(quarter * 32) << 16) + col0;
      // the parts of a long segment, added in the other accumulator
      const int ksteps = ksteps_of(it), part_stages = part_of(ksteps);
      const bool in_parts = ksteps > part_stages;
      bool got = true;
      for (int ks = 0; got && in_parts && ks < ksteps; ks += part_stages) {
        got = wait_full();
        for (int c = 0; got && c < kTile / 2; c += 32) {
          float v[32];
          mx::tmem_load32(tlane + acc * kTile + c, v);
          if (ks > 0) {
            float u[32];
            mx::tmem_load32(tlane + (acc ^ 1) * kTile + c, u);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = u[j] + v[j];
          }
          tmem_st32(tlane + (acc ^ 1) * kTile + c, v);
        }
        tmem_wait_st();
        if (got) release(acc);
      }
      if (!in_parts && !empty) got = wait_full();
      if (!got) break;
      if (in_parts) acc ^= 1;   // where the sum is
      const uint32_t tbase = tmem + ((uint32_t)(quarter * 32) << 16) + acc * kTile;
      if (!wgrad(kMode)) {
        // A lane is an output feature, a column a row of y.  Neighbouring lanes
        // exchange halves, so that an even lane has two features of the even rows,
        // an odd one of the odd rows: half the stores and addresses.
        const int odd = lane & 1;
        const size_t step = 4 * (size_t)F;   // bytes of two rows
        for (int n = 0; n < kGroups * kTile / 2; n += 32) {
          const int g = n / (kTile / 2), c = col0 + n % (kTile / 2);
          const int feat = (it.b * kGroups + g) * kTile + (int)rank * 128 + quarter * 32 + (lane & ~1);
          if (c >= it.rows) continue;   // the same for the whole warp
          float v[32];
          mx::tmem_load32(tbase + g * kTile + c, v);
          uint8_t* out = reinterpret_cast<uint8_t*>(args.out) + 2 * ((size_t)(it.row0 + c + odd) * F + feat);
          const int left = feat < F ? it.rows - c - odd : 0;   // rows from this lane's first on
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const uint32_t p = pack2(v[j], v[j + 1]), q = pack2(v[j + 2], v[j + 3]);
            const uint32_t got = __shfl_xor_sync(0xffffffffu, __byte_perm(p, q, odd ? 0x5410 : 0x7632), 1);
            const uint32_t lo = __byte_perm(p, got, odd ? 0x3254 : 0x5410), hi = __byte_perm(q, got, odd ? 0x3276 : 0x7610);
            if (j < left) *reinterpret_cast<uint32_t*>(out) = lo;
            if (j + 2 < left) *reinterpret_cast<uint32_t*>(out + step) = hi;
            out += 2 * step;
          }
          __syncwarp();   // the next columns are loaded by the whole warp
        }
      } else {
        Item ahead = it;
        if (kMode == kWgradAdd && item + pairs < total) ahead = item_of<kMode>(args, seg, item + pairs);
        const int columns = blocks_of(it) * 32;   // the same for the whole warp
        // (kWgradAdd counts every block, for the requests)
        for (int c = 0; c < (kMode == kWgradAdd ? kTile / 2 : columns); c += 4 * per) {
          if (kMode == kWgradAdd && c >= columns) {
            cp_async_wait<1>();
            if (item + pairs < total && c >= 64) request_add(ahead, (c >> 5) - 2);
            else cp_async_commit();
            continue;
          }
          float v[32] = {};
          if (!empty) mx::tmem_load32(tbase + col0 + c, v);
          if (!args.fp32) {
            float u[32] = {};
            if (!empty) mx::tmem_load32(tbase + col0 + c + 32, u);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(pack2(v[2 * j], v[2 * j + 1]));
#pragma unroll
            for (int j = 0; j < 16; ++j) v[16 + j] = __uint_as_float(pack2(u[2 * j], u[2 * j + 1]));
          }
          transpose4(v, lane);
          if (kMode == kWgradAdd) {
            const int block = c >> 5;
            cp_async_wait<1>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = (lane & ~3) + j, ch = 2 * (lane & 3);
              const uint8_t* row = adds + (warp - 2) * 2 * kAddBlock + (block & 1) * kAddBlock + r * 128;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float4 d = *reinterpret_cast<const float4*>(row + (((ch + h) ^ ((r >> 2) & 1)) << 4));
                v[8 * j + 4 * h] += d.x;
                v[8 * j + 4 * h + 1] += d.y;
                v[8 * j + 4 * h + 2] += d.z;
                v[8 * j + 4 * h + 3] += d.w;
              }
            }
            __syncwarp();
            // (add may be out: a block is read two before it is written, by the same warp)
            if (block < 2)
              request_add(it, block + 2);
            else if (item + pairs < total)
              request_add(ahead, block - 2);
            else
              cp_async_commit();
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (m0 + j < args.g.K && nl + c < F) {
              uint8_t* o = reinterpret_cast<uint8_t*>(args.out) + (at + c + (size_t)j * F) * (args.fp32 ? 4 : 2);
              const uint32_t* w = reinterpret_cast<const uint32_t*>(v + 8 * j);
              if (args.fp32 || nl + c + 8 < F)
                store8(o, wide, w);
              else
                __stcs(reinterpret_cast<uint4*>(o), make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          __syncwarp();   // the next columns are loaded by the whole warp
        }
      }
      if (empty) continue;
      release(acc);
      if (kGroups == 1) acc ^= 1;
    }
  }

  if (kMode == kWgradAdd) cp_async_wait<0>();   // (a wait that ran out left some in flight)
  tc_fence_before();
  __syncthreads();
  // Nothing targets either CTA's shared memory from here on (pipeline_end.h; the
  // same steps as end_pair, with the requests of several warps).
  {
    volatile int no_abort = 0;
    const int gave_up = s_abort;
    const uint32_t there = mapa_shared(smem_u32(const_cast<PartsEnd*>(&s_peer)), lead ? 1 : 0);
    if (threadIdx.x == 0 && gave_up) store_cluster(there + 4 * kMostParts, 1);
    __syncwarp();
    cluster_sync();   // also: neither CTA issues anything from here on
    if (gave_up || s_peer.gave_up) {   // the same in every thread of both CTAs
      if (threadIdx.x == 0)
        for (int w = 0; w < kParts; ++w) store_cluster(there + 4 * w, s_end.issued[w]);
      __syncwarp();
      cluster_sync();
      if (threadIdx.x == 0) {
        int mine[kParts], peer[kParts];
        for (int w = 0; w < kParts; ++w) mine[w] = s_end.issued[w], peer[w] = s_peer.issued[w];
        settle_pair_parts(
            lead, mine, peer, parts, kStages, [&](int i) { mbar_complete_tx(full0 + 8 * (i % kStages), s_tx[i % kStages]); },
            [&](int i) { mbar_arrive_expect_tx_remote(mapa_shared(full0 + 8 * (i % kStages), 0), s_tx[i % kStages]); });
        if (lead)
          wait_pair_parts(mine, peer, parts, kStages, [&](int st, uint32_t parity) {
            mbar_wait_cluster(full0 + 8 * st, parity, &no_abort);
          });
      }
      __syncwarp();
      cluster_sync();
    }
    if (threadIdx.x == 0) mbar_wait_cluster(drain, 0, &no_abort);
    __syncwarp();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ------------------------------------------------------------------ host
bool encode(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [outer][rows][cols] in boxes of box_rows rows and 64 columns.
bool map_rows(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows,
              uint64_t outer, uint32_t box_rows) {
  const cuuint64_t dims[3] = {cols, rows, outer}, strides[2] = {2 * cols, 2 * cols * rows};
  const cuuint32_t box[3] = {64, box_rows, 1};
  return encode(fn, m, base, outer ? 3 : 2, dims, strides, box);
}

// The same tensor as [outer][cols / 64][rows][64], 64 rows and 128 columns a
// box: an MN-major operand's two halves in one request.
bool map_wide(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows,
              uint64_t outer) {
  const cuuint64_t dims[4] = {64, rows, cols / 64, outer}, strides[3] = {2 * cols, 128, 2 * cols * rows};
  const cuuint32_t box[4] = {64, kBK, 2, 1};
  return encode(fn, m, base, outer ? 4 : 3, dims, strides, box);
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
int resident_pairs(int sms, int threads) {
  static int cache[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
  cudaFuncSetAttribute(grouped_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<kMode>::kSmemBytes);
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)(sms / 2), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = Cfg<kMode>::kSmemBytes;
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
  const bool gathers = wgrad(kMode) || a.gather_b;
  const int cap = resident_pairs<kMode>(sms, Cfg<kMode>::kMaxThreads);
  a.pairs = (int)(items < cap ? items : cap);
  launch_pdl(grouped_kernel<kMode>, dim3(2 * a.pairs), dim3(gathers ? Cfg<kMode>::kMaxThreads : kThreads), Cfg<kMode>::kSmemBytes, s, m, a);
}

// The rows that experts hold in all, at most.
long long routes_of(const GroupArgs& g) {
  const long long r = (long long)g.T * g.slots;
  return r < g.max_rows ? r : g.max_rows;
}

// Whether a product's items have two groups of 256 features.  They request a
// row tile once for both, but keep one accumulator, whose stores nothing overlaps,
// and leave the last wave of items emptier.  The time of a wave of double items
// over that of two waves of single ones was 0.94 for gathered rows (whose requests
// bound: W2's input gradient of 4096 tokens in the 8-expert layer 612 -> 577 us),
// 0.98 for rows in place (W13's product of 8192 tokens in the 128-expert layer 292
// -> 281; 0.94 to 1.06, the latter in the 8-expert layer), 0.9 where experts average
// at most 128 rows (W13 of 64 tokens in the 128-expert layer 122 -> 116); the waves
// follow from the tiles to be expected: at least one an expert, half of its last one
// filled.
bool wide_items(const GroupArgs& g, bool gather, int sms) {
  const double routes = (double)routes_of(g), experts = routes < g.N ? routes : g.N;
  const double tiles = std::fmax(routes / kTile + 0.5 * experts, experts), units = sms / 2;
  const double one = std::ceil(tiles * ((g.F + kTile - 1) / kTile) / units);
  const double two = std::ceil(tiles * ((g.F + 2 * kTile - 1) / (2 * kTile)) / units);
  return 2.0 * two * (routes <= 128.0 * g.N ? 0.9 : gather ? 0.94 : 0.98) < one;
}

}  // namespace

bool launch_grouped_gemm(const GroupedGemmArgs& in, PFN_cuTensorMapEncodeTiled_v12000 fn, int sms, cudaStream_t s) {
  const GroupArgs& g = in.g;
  const uint64_t K = g.K, F = g.F, N = g.N, rows = in.gather ? (uint64_t)g.T : (uint64_t)g.max_rows;
  Maps m{};
  Args a{};
  a.wide_a = !in.transposed && F % 64 == 0;
  if (!(in.transposed ? map_rows(fn, &m.a, in.w, K, F, N, 128)
        : a.wide_a    ? map_wide(fn, &m.a, in.w, F, K, N)
                      : map_rows(fn, &m.a, in.w, F, K, N, kBK)) ||
      (in.gather && !map_rows(fn, &m.b_rows, in.x, K, rows, 0, 1)))
    return false;
  for (int i = 0; i < 4 && !in.gather; ++i)
    if (!map_rows(fn, &m.b_box[i], in.x, K, rows, 0, 16 << i)) return false;
  a.g = g;
  a.gather_b = in.gather;
  set_divisor(a, (uint32_t)g.slots);
  a.out = in.y;
  a.na = 1;
  const long long routes = routes_of(g), tiles = routes / kTile + (routes < g.N ? routes : g.N);
  const bool wide = wide_items(g, in.gather, sms);
  a.nb = wide ? (g.F + 2 * kTile - 1) / (2 * kTile) : (g.F + kTile - 1) / kTile;
  if (wide && in.transposed)
    launch<kGemmTransposedWide>(m, a, tiles * a.nb, sms, s);
  else if (wide)
    launch<kGemmWide>(m, a, tiles * a.nb, sms, s);
  else if (in.transposed)
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
  Args a{};
  a.wide_a = K % 64 == 0;
  a.wide_b = F % 64 == 0;
  auto maps_of = [&](const uint16_t* p, uint64_t cols, uint64_t rows, bool gather, bool wide, CUtensorMap* box,
                     CUtensorMap* small, CUtensorMap* one) {
    if (!map_rows(fn, one, p, cols, rows, 0, 1)) return false;
    return gather || ((wide ? map_wide(fn, box, p, cols, rows, 0) : map_rows(fn, box, p, cols, rows, 0, kBK)) &&
                      map_rows(fn, small, p, cols, rows, 0, kRowBox));
  };
  if (!maps_of(in.x, K, xr, in.gather_x, a.wide_a, &m.a, &m.a_small, &m.a_rows) ||
      !maps_of(in.dy, F, dr, in.gather_dy, a.wide_b, &m.b, &m.b_small, &m.b_rows))
    return false;
  a.g = g;
  a.gather_a = in.gather_x;
  a.gather_b = in.gather_dy;
  set_divisor(a, (uint32_t)g.slots);
  a.add = in.add;
  a.out = in.dw;
  a.fp32 = in.fp32;
  a.wide_out = reinterpret_cast<uintptr_t>(in.dw) % 32 == 0 && (in.fp32 || g.F % 16 == 0);
  a.na = (g.K + kTile - 1) / kTile;
  a.nb = (g.F + kTile - 1) / kTile;
  if (in.add)
    launch<kWgradAdd>(m, a, (long long)g.N * a.na * a.nb, sms, s);
  else
    launch<kWgrad>(m, a, (long long)g.N * a.na * a.nb, sms, s);
  return true;
}

}  // namespace moe
