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
  int tile_rows;             // token rows of a tile of the list: kMxTileRows, or twice that (CTA pairs)
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
// Token rows of a tile: 256 (CTA pairs) or 128.  max_rows: routed rows at most.
int mx_tile_rows(int64_t max_rows, int experts);
// Weight rows of a work item: a rule on the number of items (see the definition).
int mx_tile_features(int tile_rows, int features, int64_t max_tiles, int sms);
void launch_mx_gemm(bool w13, const MxMaps& m, const MxGemmArgs& a, int64_t max_tiles, int sms, cudaStream_t s);

// Routed rows of the activations in tile order: codes [rows, H/2] and scales
// [128-row tile][H/128][512] (identity_T > 0: the scales alone, rows 0..T-1).
void launch_mx_gather(const uint8_t* codes, const uint8_t* scales, const int32_t* sorted_route_ids, int slots,
                      int T, int H, const GemmTile* tiles, const int32_t* num_tiles, int tile_rows, int identity_T,
                      int64_t max_tiles, uint8_t* x_perm, uint8_t* x_sf, cudaStream_t s);

}  // namespace moe
