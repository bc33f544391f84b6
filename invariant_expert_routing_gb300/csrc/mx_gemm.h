// Grouped SwiGLU expert GEMMs on microscaled 4-bit operands: launch arguments.
// Internal, not part of the C ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "gemm.h"

namespace moe {

constexpr int kMxTileRows = 128;   // token rows of a CTA's tile; a pair's tile has 256

struct MxGemmArgs {
  int K;                     // reduction length (H for W13, I for W2)
  int features;              // weight rows of one expert (2I or H)
  int tile_rows;             // token rows of a tile of the list: 256 (CTA pairs), 128, or 32 (operands swapped)
  int tile_features;         // weight rows of one work item
  const GemmTile* tiles;     // tile list on the device
  const int32_t* num_tiles;  // device count
  int identity_T;            // > 0: rows 0..T-1 of one expert, no tile list (shared expert)
  const uint8_t* a_sf;       // activation scales [128-row tile][K/128][512]
  const uint8_t* b_sf;       // weight scales [expert][features/128][K/128][512]
  uint8_t* out_codes;        // W13: codes [rows, I/2]
  uint8_t* out_sf;           // W13: scales [128-row tile][I/128][512]
  uint16_t* out;             // W2: bf16 [rows, H]
  int out_ld;                // I or H
  int* status;
  int concurrent;            // work units resident at once (set by the launcher)
  unsigned long long wait_ns;
};

// w: W13 5-D (K bytes, 32 rows, gate/up, 32-feature block, expert), W2 3-D (K
// bytes, row, expert); x / x_small: activation codes, boxes of 128 and 32 rows.
// CTA pairs also take the scales, as rows of one 512-byte chunk, boxes of two
// (sfa, sfb), and the W2 output, boxes of 32 rows x 64 columns (y); their W13 box
// is one run of 32 rows.
struct MxMaps {
  CUtensorMap w, x, x_small, sfa, sfb, y;
};

bool mx_gemm_smem_ok();
// Token rows of a tile: 256 (CTA pairs), 128, or 32 (operands swapped), by the
// average number of rows an expert has.
int mx_tile_rows(int64_t rows, int experts);
int64_t mx_swap_max_rows(int experts);   // the most rows with 32-row tiles
// Weight rows of a work item: a rule on the number of items (tiles: as expected).
int mx_tile_features(int tile_rows, int features, int64_t tiles, int sms);
void launch_mx_gemm(bool w13, const MxMaps& m, const MxGemmArgs& a, int64_t max_tiles, int sms, cudaStream_t s);

// The launch before the GEMMs: the tile list (tile_rows rows), and the
// activations in tile order: codes [rows, H/2] and scales [tile][H/128][512],
// a tile of 256 rows as two of 128.  identity_T > 0: the scales of rows
// 0..T-1 alone.
struct MxFrontArgs {
  const uint8_t *codes, *scales;   // [T, H/2], [T, H/32]
  const int32_t *sorted, *block_expert, *num_padded;
  int T, slots, H, N, B, tile_rows, identity_T;
  int64_t max_rows, max_tiles;
  GemmTile* tiles;
  int32_t* num_tiles;
  uint8_t *x_perm, *x_sf;
  int* status;
  const uint8_t* w13;              // W13 codes [N, 2I, H/2]: the first of them are prefetched
  int I;
  int scale_ctas, code_ctas;       // CTAs that place scales and copy codes (set by the launcher)
  int prefetch_units;              // 32 features of W13 each (set by the launcher)
};
void launch_mx_front(const MxFrontArgs& a, int sms, cudaStream_t s);

}  // namespace moe
