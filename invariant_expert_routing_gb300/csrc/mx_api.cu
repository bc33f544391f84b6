// C ABI of the 4-bit expert path (include/moe_api.h): residual + norm,
// routing by scores, microscaled 4-bit conversion, the grouped expert FFN on
// 4-bit operands and the pre-norm block that runs them together.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api_internal.h"
#include "kernels.h"
#include "mx_gemm.h"

namespace {

using moe::GemmTile;
namespace api = moe::api;

constexpr int kSfBlock = 32;      // elements per scale
constexpr int kMaxHidden = 32768;

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Bytes of the scale chunks of `tiles` 128-row tiles with K elements a row.
size_t sf_bytes(int64_t tiles, int K) { return (size_t)tiles * moe::kMxTileRows * (K / kSfBlock); }

// 128-row scale tiles under a tile of the list.
int64_t scale_tiles(int tile_rows) { return tile_rows > moe::kMxTileRows ? tile_rows / moe::kMxTileRows : 1; }

// Rows that hold a route (at most, with a capacity): what the experts average.
// With expert choice a token has a slot for every expert but the experts take
// `capacity` tokens each.
int64_t routed_rows(const moe_config* c, int32_t T) {
  if (c->routing == MOE_ROUTING_EXPERT_CHOICE) return (int64_t)c->num_experts * api::capacity(c, T);
  return (int64_t)T * c->top_k;
}

int tile_rows_of(const moe_config* c, int32_t T) { return moe::mx_tile_rows(routed_rows(c, T), c->num_experts); }

// The most tokens up to T that run with 32-row tiles.
int32_t swap_tokens(const moe_config* c, int32_t T) {
  int32_t lo = 0, hi = T;
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo + 1) / 2;
    if (routed_rows(c, mid) <= moe::mx_swap_max_rows(c->num_experts))
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Workspace regions, each 256-byte aligned; the status word is at offset 0.
struct Layout {
  size_t status, tiles, num_tiles, x_perm, x_sf, a, a_sf, x_sh_sf, a_sh, a_sh_sf,
      // moe_forward_mx alone
      residual, norm, codes, scales, logits, rpart, topk, gates, kept, pos, rank, tile_count, seg_off, sorted, blocks,
      num_padded, counts, dropped, y, y_sh, total;
};

Layout layout_of(const moe_config* c, int32_t T) {
  const size_t N = c->num_experts, H = c->hidden, I = c->intermediate, Is = c->shared_intermediate;
  const size_t R = (size_t)T * api::slots(c), rows = (size_t)api::max_rows(c, T);
  // The tile height follows the number of routed rows; the regions hold the list
  // and the scale tiles of any height that up to T tokens may take, so that a
  // workspace for T serves every smaller call.
  const int64_t tiles = std::max(api::max_tiles(c, swap_tokens(c, T), 32), api::max_tiles(c, T, moe::kMxTileRows));
  const int64_t sf_tiles = std::max(tiles, 2 * api::max_tiles(c, T, 2 * moe::kMxTileRows));
  const int64_t tiles_t = 2 * (((int64_t)T + 2 * moe::kMxTileRows - 1) / (2 * moe::kMxTileRows));
  Layout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = round_up(off + bytes, 256);
    return at;
  };
  L.status = take(sizeof(int32_t));
  L.tiles = take(sizeof(GemmTile) * (size_t)tiles);
  L.num_tiles = take(2 * sizeof(int32_t));
  // the activations keep one tile of rows of slack so that every tile load stays inside them
  L.x_perm = take((rows + moe::kMxTileRows) * H / 2);
  L.x_sf = take(sf_bytes(sf_tiles, (int)H));
  L.a = take((rows + moe::kMxTileRows) * I / 2);
  L.a_sf = take(sf_bytes(sf_tiles, (int)I));
  L.x_sh_sf = take(Is ? sf_bytes(tiles_t, (int)H) : 0);
  L.a_sh = take(Is ? ((size_t)T + moe::kMxTileRows) * Is / 2 : 0);
  L.a_sh_sf = take(Is ? sf_bytes(tiles_t, (int)Is) : 0);
  L.residual = take(2 * (size_t)T * H);
  L.norm = take(2 * (size_t)T * H);
  L.codes = take((size_t)T * H / 2);
  L.scales = take((size_t)T * H / kSfBlock);
  L.logits = take(sizeof(float) * (size_t)T * N);
  L.rpart = take(sizeof(float) * moe::chunked_router_part_floats(T, (int)H, (int)N));
  L.topk = take(sizeof(int32_t) * R);
  L.gates = take(sizeof(float) * R);
  L.kept = take(R);
  L.pos = take(sizeof(int32_t) * R);
  L.rank = take(sizeof(int32_t) * R);
  L.tile_count = take(sizeof(int32_t) * ((R + moe::kDispatchTile - 1) / moe::kDispatchTile) * N);
  L.seg_off = take(sizeof(int32_t) * N);
  L.sorted = take(sizeof(int32_t) * rows);
  L.blocks = take(sizeof(int32_t) * (size_t)api::max_blocks(c, T));
  L.num_padded = take(sizeof(int32_t));
  L.counts = take(sizeof(int32_t) * N);
  L.dropped = take(sizeof(int32_t));
  L.y = take(2 * rows * H);
  L.y_sh = take(Is ? 2 * (size_t)T * H : 0);
  L.total = off;
  return L;
}

template <class P>
P* at(void* ws, size_t off) {
  return reinterpret_cast<P*>(static_cast<char*>(ws) + off);
}

moe_status check_ws(const moe_config* c, int32_t T, const void* ws, size_t ws_bytes) {
  MOE_TRY(api::need(ws));
  return ws_bytes < layout_of(c, T).total ? MOE_ERR_WORKSPACE : MOE_OK;
}

moe_status check_scoring(const moe_config* c, const moe_scoring* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->score != MOE_SCORE_SOFTMAX && s->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (s->group_score != MOE_GROUP_MAX && s->group_score != MOE_GROUP_TOP2_SUM) return MOE_ERR_INVALID_ARG;
  if (s->renormalize != 0 && s->renormalize != 1) return MOE_ERR_INVALID_ARG;
  if (!std::isfinite(s->scale) || s->scale < 0.0f) return MOE_ERR_INVALID_ARG;
  if (c->routing != MOE_ROUTING_TOKEN_CHOICE) return MOE_ERR_INVALID_ARG;
  const int N = c->num_experts;
  const int groups = s->num_groups == 0 ? 1 : s->num_groups;
  const int top = s->top_groups == 0 ? groups : s->top_groups;
  if (groups < 1 || top < 1 || top > groups || N % groups) return MOE_ERR_INVALID_ARG;
  if (groups > moe::route_scored_max_groups()) return MOE_ERR_UNSUPPORTED;
  if (groups > 1 && s->group_score == MOE_GROUP_TOP2_SUM && N / groups < 2) return MOE_ERR_INVALID_ARG;
  if (c->top_k > top * (N / groups)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status route_impl(const moe_config* c, const moe_scoring* s, int32_t T, const float* logits,
                      const float* score_bias, int32_t* idx, float* gate, cudaStream_t st) {
  const int groups = s->num_groups == 0 ? 1 : s->num_groups;
  const int top = s->top_groups == 0 ? groups : s->top_groups;
  moe::launch_route_scored(logits, score_bias, T, c->num_experts, c->top_k, s->score == MOE_SCORE_SIGMOID,
                           top == groups ? 1 : groups, top, s->group_score == MOE_GROUP_TOP2_SUM, s->renormalize != 0,
                           s->scale == 0.0f ? 1.0f : s->scale, idx, gate, st);
  return api::last_error();
}

// ----------------------------------------------------------------- tensor maps
bool encode(CUtensorMap* m, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base, int rank,
            const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  auto fn = api::tensor_map_encode();
  if (!fn) return false;
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, type, rank, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Bytes with 128-byte swizzle, 128 of them (256 elements of K) a box.
bool encode_codes(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                  const cuuint32_t* box) {
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, base, rank, dims, strides, box);
}

// Scale chunks as rows of 512 bytes, two a box.
bool map_scales(CUtensorMap* m, const void* base, uint64_t chunks) {
  const cuuint64_t dims[2] = {128, chunks}, strides[1] = {512};
  const cuuint32_t box[2] = {128, 2};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, CU_TENSOR_MAP_SWIZZLE_NONE, base, 2, dims, strides, box);
}

// bf16 output rows, 32 rows x 64 columns a box.
bool map_out(CUtensorMap* m, const void* base, uint64_t H, uint64_t rows) {
  const cuuint64_t dims[2] = {H, rows}, strides[1] = {2 * H};
  const cuuint32_t box[2] = {64, 32};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B, base, 2, dims, strides, box);
}

bool map_rows(CUtensorMap* m, const void* base, int K, uint64_t rows, uint32_t box_rows) {
  const cuuint64_t pitch = (cuuint64_t)K / 2;
  const cuuint64_t dims[2] = {pitch, rows}, strides[1] = {pitch};
  const cuuint32_t box[2] = {128, box_rows};
  return encode_codes(m, base, 2, dims, strides, box);
}

// W13 [N, 2I, K/2]: (byte, row of a 32-feature block, gate/up, block, expert),
// so that one box holds 32 gate and the same 32 up rows in turns (box_rows 32:
// one such run).
bool map_w13(CUtensorMap* m, const void* base, int K, int I, int N, int box_rows) {
  const cuuint64_t pitch = (cuuint64_t)K / 2;
  const cuuint64_t dims[5] = {pitch, 32, 2, (cuuint64_t)I / 32, (cuuint64_t)N};
  const cuuint64_t strides[4] = {pitch, pitch * I, pitch * 32, pitch * 2 * I};
  const cuuint32_t box[5] = {128, 32, box_rows == 32 ? 1u : 2u, box_rows == 32 ? 1u : (cuuint32_t)box_rows / 64, 1};
  return encode_codes(m, base, 5, dims, strides, box);
}

// W2 [N, H, I/2]: (byte, row, expert); rows past an expert's last read as zeros.
bool map_w2(CUtensorMap* m, const void* base, int K, int H, int N, int box_rows) {
  const cuuint64_t pitch = (cuuint64_t)K / 2;
  const cuuint64_t dims[3] = {pitch, (cuuint64_t)H, (cuuint64_t)N}, strides[2] = {pitch, pitch * H};
  const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
  return encode_codes(m, base, 3, dims, strides, box);
}

// ----------------------------------------------------------------- expert FFN
// The two GEMMs of one set of experts: activations x (codes, tile-order
// scales) -> a (codes, tile-order scales) -> y.
moe_status gemms(const moe_config* c, int H, int I, int N, const uint8_t* x, const uint8_t* x_sf, uint64_t x_rows,
                 const uint8_t* w13, const uint8_t* w13_sf, const uint8_t* w2, const uint8_t* w2_sf, uint8_t* a,
                 uint8_t* a_sf, uint64_t a_rows, uint16_t* y, uint64_t y_rows, const GemmTile* tiles,
                 const int32_t* num_tiles, int tile_rows, int identity_T, int64_t max_tiles, int64_t tiles_expected,
                 int sms, int* status, cudaStream_t s) {
  const bool pair = tile_rows > moe::kMxTileRows;
  const int f13 = moe::mx_tile_features(tile_rows, 2 * I, tiles_expected, sms);
  const int f2 = moe::mx_tile_features(tile_rows, H, tiles_expected, sms);
  const uint64_t sf_tiles = (uint64_t)max_tiles * scale_tiles(tile_rows);
  const uint32_t box = 128, box_small = 32;   // token rows
  moe::MxMaps m13, m2;
  // a CTA of a pair loads half of the weight rows of an item
  if (!map_w13(&m13.w, w13, H, I, N, pair ? 32 : f13) || !map_rows(&m13.x, x, H, x_rows, box) ||
      !map_rows(&m13.x_small, x, H, x_rows, box_small) || !map_w2(&m2.w, w2, I, H, N, pair ? f2 / 2 : f2) ||
      !map_rows(&m2.x, a, I, a_rows, box) || !map_rows(&m2.x_small, a, I, a_rows, box_small))
    return MOE_ERR_CUDA;
  if (pair && (!map_scales(&m13.sfa, x_sf, sf_tiles * (H / 128)) || !map_scales(&m2.sfa, a_sf, sf_tiles * (I / 128)) ||
               !map_scales(&m13.sfb, w13_sf, (uint64_t)N * (2 * I / 128) * (H / 128)) ||
               !map_scales(&m2.sfb, w2_sf, (uint64_t)N * (H / 128) * (I / 128)) || !map_out(&m2.y, y, H, y_rows)))
    return MOE_ERR_CUDA;
  if (pair) m13.y = m2.y;
  moe::MxGemmArgs g{};
  g.K = H;
  g.features = 2 * I;
  g.tile_rows = tile_rows;
  g.tile_features = f13;
  g.tiles = tiles;
  g.num_tiles = num_tiles;
  g.identity_T = identity_T;
  g.a_sf = x_sf;
  g.b_sf = w13_sf;
  g.out_codes = a;
  g.out_sf = a_sf;
  g.out_ld = I;
  g.status = status;
  g.wait_ns = (unsigned long long)c->debug_wait_ns;
  moe::launch_mx_gemm(true, m13, g, max_tiles, sms, s);
  g.K = I;
  g.features = H;
  g.tile_features = f2;
  g.a_sf = a_sf;
  g.b_sf = w2_sf;
  g.out = y;
  g.out_ld = H;
  moe::launch_mx_gemm(false, m2, g, max_tiles, sms, s);
  return api::last_error();
}

struct Experts {
  const uint8_t *w13, *w13_sf, *w2, *w2_sf, *w13s, *w13s_sf, *w2s, *w2s_sf;
};

moe_status check_experts(const moe_config* c, const Experts& w) {
  MOE_TRY(api::need(w.w13));
  MOE_TRY(api::need(w.w13_sf));
  MOE_TRY(api::need(w.w2));
  MOE_TRY(api::need(w.w2_sf));
  if (c->shared_intermediate > 0) {
    MOE_TRY(api::need(w.w13s));
    MOE_TRY(api::need(w.w13s_sf));
    MOE_TRY(api::need(w.w2s));
    MOE_TRY(api::need(w.w2s_sf));
  }
  return MOE_OK;
}

moe_status ffn_impl(const moe_config* c, int32_t T, const uint8_t* codes, const uint8_t* scales, const Experts& w,
                    const int32_t* sorted, const int32_t* blocks, const int32_t* num_padded, uint16_t* y_perm,
                    uint16_t* y_shared, void* ws, cudaStream_t s) {
  const Layout L = layout_of(c, T);
  const int H = c->hidden, I = c->intermediate, N = c->num_experts, slots = api::slots(c);
  const int64_t rows = api::max_rows(c, T);
  const int64_t routed = routed_rows(c, T);
  const int tile_rows = tile_rows_of(c, T);
  const int64_t max_tiles = api::max_tiles(c, T, tile_rows);
  const int sms = api::sm_count();
  if (sms <= 0 || !moe::mx_gemm_smem_ok()) return MOE_ERR_CUDA;
  moe::MxFrontArgs f{};
  f.codes = codes;
  f.scales = scales;
  f.sorted = sorted;
  f.block_expert = blocks;
  f.num_padded = num_padded;
  f.T = T;
  f.slots = slots;
  f.H = H;
  f.N = N;
  f.B = c->block_size;
  f.tile_rows = tile_rows;
  f.max_rows = rows;
  f.max_tiles = max_tiles;
  f.tiles = at<GemmTile>(ws, L.tiles);
  f.num_tiles = at<int32_t>(ws, L.num_tiles);
  f.x_perm = at<uint8_t>(ws, L.x_perm);
  f.x_sf = at<uint8_t>(ws, L.x_sf);
  f.w13 = w.w13;
  f.I = I;
  f.status = at<int>(ws, L.status);
  moe::launch_mx_front(f, sms, s);
  const uint64_t perm_rows = (uint64_t)rows + moe::kMxTileRows;
  // tiles as they come: one for each expert that routes can touch, and the full ones
  const int64_t expected = std::min<int64_t>(routed, N) + routed / tile_rows;
  MOE_TRY(gemms(c, H, I, N, f.x_perm, f.x_sf, perm_rows, w.w13, w.w13_sf, w.w2, w.w2_sf, at<uint8_t>(ws, L.a),
                at<uint8_t>(ws, L.a_sf), perm_rows, y_perm, (uint64_t)rows, f.tiles, f.num_tiles, tile_rows, 0, max_tiles,
                expected, sms, f.status, s));
  if (c->shared_intermediate > 0) {
    moe::MxFrontArgs g{};
    g.codes = codes;
    g.scales = scales;
    g.T = T;
    g.slots = 1;
    g.H = H;
    g.tile_rows = moe::mx_tile_rows(T, 1);
    g.identity_T = T;
    g.max_tiles = ((int64_t)T + g.tile_rows - 1) / g.tile_rows;
    g.x_sf = at<uint8_t>(ws, L.x_sh_sf);
    moe::launch_mx_front(g, sms, s);
    MOE_TRY(gemms(c, H, c->shared_intermediate, 1, codes, g.x_sf, (uint64_t)T, w.w13s, w.w13s_sf, w.w2s, w.w2s_sf,
                  at<uint8_t>(ws, L.a_sh), at<uint8_t>(ws, L.a_sh_sf), (uint64_t)T + moe::kMxTileRows, y_shared, (uint64_t)T,
                  nullptr, nullptr, g.tile_rows, T, g.max_tiles, g.max_tiles, sms, f.status, s));
  }
  return api::last_error();
}

moe_status check_norm(int32_t T, int32_t H, float eps) {
  if (T < 0 || H <= 0 || !(eps >= 0.0f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if (H % kSfBlock || H > kMaxHidden || T > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_mx(int64_t rows, int32_t K) {
  if (rows < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (K % kSfBlock || rows > ((int64_t)1 << 40) / K) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_check_scoring(const moe_config* cfg, const moe_scoring* scoring) {
  MOE_TRY(api::check_config(cfg));
  return check_scoring(cfg, scoring);
}

moe_status moe_route_scored(const moe_config* cfg, const moe_scoring* scoring, int32_t T, const float* logits,
                            const float* score_bias, int32_t* topk_idx, float* topk_gate, void* stream) {
  MOE_TRY(api::check_config(cfg));
  MOE_TRY(api::check_tokens(cfg, T));
  MOE_TRY(check_scoring(cfg, scoring));
  if (T == 0) return MOE_OK;
  MOE_TRY(api::need(logits));
  MOE_TRY(api::optional(score_bias));
  MOE_TRY(api::need(topk_idx));
  MOE_TRY(api::need(topk_gate));
  return route_impl(cfg, scoring, T, logits, score_bias, topk_idx, topk_gate, static_cast<cudaStream_t>(stream));
}

moe_status moe_add_norm(int32_t T, int32_t H, const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                        float eps, uint16_t* residual_out, uint16_t* out, uint8_t* codes, uint8_t* scales,
                        void* stream) {
  MOE_TRY(check_norm(T, H, eps));
  if (T == 0) return MOE_OK;
  MOE_TRY(api::need(x));
  MOE_TRY(api::optional(residual));
  MOE_TRY(api::need(weight));
  MOE_TRY(api::optional(residual_out));
  MOE_TRY(api::optional(out));
  MOE_TRY(api::optional(codes));
  MOE_TRY(api::optional(scales));
  if ((codes == nullptr) != (scales == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!out && !codes) return MOE_ERR_INVALID_ARG;
  const int sms = api::sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  moe::launch_add_norm(x, residual, weight, eps, T, H, residual_out, out, codes, scales, sms,
                       static_cast<cudaStream_t>(stream));
  return api::last_error();
}

moe_status moe_quantize_mx(int64_t rows, int32_t K, const uint16_t* x, uint8_t* codes, uint8_t* scales,
                           void* stream) {
  MOE_TRY(check_mx(rows, K));
  if (rows == 0) return MOE_OK;
  MOE_TRY(api::need(x));
  MOE_TRY(api::need(codes));
  MOE_TRY(api::need(scales));
  moe::launch_quantize_mx(x, (size_t)rows * K, codes, scales, static_cast<cudaStream_t>(stream));
  return api::last_error();
}

moe_status moe_dequantize_mx(int64_t rows, int32_t K, const uint8_t* codes, const uint8_t* scales, uint16_t* out,
                             void* stream) {
  MOE_TRY(check_mx(rows, K));
  if (rows == 0) return MOE_OK;
  MOE_TRY(api::need(codes));
  MOE_TRY(api::need(scales));
  MOE_TRY(api::need(out));
  moe::launch_dequantize_mx(codes, scales, (size_t)rows * K, out, static_cast<cudaStream_t>(stream));
  return api::last_error();
}

moe_status moe_quantize_weights_mx(int32_t experts, int32_t K, int32_t F, const uint16_t* w, uint8_t* codes,
                                   uint8_t* scales, void* stream) {
  if (experts < 0 || F <= 0) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_mx(experts, K));
  if (F % 8 || F > (1 << 21) || experts > 65535) return MOE_ERR_UNSUPPORTED;
  if (experts == 0) return MOE_OK;
  MOE_TRY(api::need(w));
  MOE_TRY(api::need(codes));
  MOE_TRY(api::need(scales));
  moe::launch_quantize_weights_mx(w, experts, K, F, codes, scales, static_cast<cudaStream_t>(stream));
  return api::last_error();
}

moe_status moe_pack_scales_mx(int32_t experts, int32_t rows, int32_t K, int32_t gate_up, const uint8_t* scales,
                              uint8_t* packed, void* stream) {
  if (experts < 0 || rows <= 0 || K <= 0 || (gate_up != 0 && gate_up != 1)) return MOE_ERR_INVALID_ARG;
  if (rows % 128 || K % 128 || rows > (1 << 18) || K > (1 << 17) || experts > 65535) return MOE_ERR_UNSUPPORTED;
  if (experts == 0) return MOE_OK;
  MOE_TRY(api::need(scales));
  MOE_TRY(api::need(packed));
  // every word moves: there is no order in which this could be done in place
  const uint8_t* end = scales + (size_t)experts * rows * (K / kSfBlock);
  if (packed < end && scales < packed + (end - scales)) return MOE_ERR_INVALID_ARG;
  moe::launch_pack_scales_mx(scales, experts, rows, K, gate_up != 0, packed, static_cast<cudaStream_t>(stream));
  return api::last_error();
}

size_t moe_workspace_bytes_mx(const moe_config* cfg, int32_t max_tokens) {
  if (api::check_config(cfg) != MOE_OK || api::check_tokens(cfg, max_tokens) != MOE_OK) return 0;
  return layout_of(cfg, max_tokens).total;
}

int32_t moe_expert_ffn_mx_tile_rows(const moe_config* cfg, int32_t T) {
  if (api::check_config(cfg) != MOE_OK || api::check_tokens(cfg, T) != MOE_OK) return 0;
  return tile_rows_of(cfg, T);
}

moe_status moe_expert_ffn_mx(const moe_config* cfg, int32_t T, const uint8_t* x_codes, const uint8_t* x_scales,
                             const uint8_t* w13, const uint8_t* w13_scales, const uint8_t* w2,
                             const uint8_t* w2_scales, const uint8_t* w13_shared, const uint8_t* w13_shared_scales,
                             const uint8_t* w2_shared, const uint8_t* w2_shared_scales,
                             const int32_t* sorted_route_ids, const int32_t* block_expert, const int32_t* num_padded,
                             uint16_t* y_perm, uint16_t* y_shared, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(api::check_config(cfg));
  MOE_TRY(api::check_tokens(cfg, T));
  if (T == 0) return MOE_OK;
  const Experts w{w13, w13_scales, w2, w2_scales, w13_shared, w13_shared_scales, w2_shared, w2_shared_scales};
  MOE_TRY(api::need(x_codes));
  MOE_TRY(api::need(x_scales));
  MOE_TRY(check_experts(cfg, w));
  MOE_TRY(api::need(sorted_route_ids));
  MOE_TRY(api::need(block_expert));
  MOE_TRY(api::need(num_padded));
  MOE_TRY(api::need(y_perm));
  if (cfg->shared_intermediate > 0) MOE_TRY(api::need(y_shared));
  MOE_TRY(check_ws(cfg, T, ws, ws_bytes));
  return ffn_impl(cfg, T, x_codes, x_scales, w, sorted_route_ids, block_expert, num_padded, y_perm, y_shared, ws,
                  static_cast<cudaStream_t>(stream));
}

moe_status moe_forward_mx(const moe_config* cfg, const moe_scoring* scoring, int32_t T, const uint16_t* x,
                          const uint16_t* residual, const uint16_t* norm_weight, float eps, const uint16_t* w_gate,
                          const float* router_bias, const float* score_bias, const uint8_t* w13,
                          const uint8_t* w13_scales, const uint8_t* w2, const uint8_t* w2_scales,
                          const uint8_t* w13_shared, const uint8_t* w13_shared_scales, const uint8_t* w2_shared,
                          const uint8_t* w2_shared_scales, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(api::check_config(cfg));
  MOE_TRY(api::check_tokens(cfg, T));
  MOE_TRY(check_scoring(cfg, scoring));
  MOE_TRY(check_norm(T, cfg->hidden, eps));
  if (cfg->overflow_policy == MOE_OVERFLOW_REROUTE && cfg->capacity_factor > 0.0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const Experts w{w13, w13_scales, w2, w2_scales, w13_shared, w13_shared_scales, w2_shared, w2_shared_scales};
  MOE_TRY(api::need(x));
  MOE_TRY(api::optional(residual));
  MOE_TRY(api::need(norm_weight));
  MOE_TRY(api::need(w_gate));
  MOE_TRY(api::optional(router_bias));
  MOE_TRY(api::optional(score_bias));
  MOE_TRY(check_experts(cfg, w));
  MOE_TRY(api::need(out));
  MOE_TRY(check_ws(cfg, T, ws, ws_bytes));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int sms = api::sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  const Layout L = layout_of(cfg, T);
  const int H = cfg->hidden, N = cfg->num_experts;
  // without a residual the layer's input is its residual stream
  uint16_t* sum = residual ? at<uint16_t>(ws, L.residual) : nullptr;
  uint16_t* norm = at<uint16_t>(ws, L.norm);
  uint8_t* codes = at<uint8_t>(ws, L.codes);
  uint8_t* scales = at<uint8_t>(ws, L.scales);
  float* logits = at<float>(ws, L.logits);
  int32_t* idx = at<int32_t>(ws, L.topk);
  float* gates = at<float>(ws, L.gates);
  uint8_t* kept = at<uint8_t>(ws, L.kept);
  int32_t* pos = at<int32_t>(ws, L.pos);
  int32_t* sorted = at<int32_t>(ws, L.sorted);
  int32_t* blocks = at<int32_t>(ws, L.blocks);
  int32_t* num_padded = at<int32_t>(ws, L.num_padded);
  uint16_t* y = at<uint16_t>(ws, L.y);
  uint16_t* y_sh = cfg->shared_intermediate ? at<uint16_t>(ws, L.y_sh) : nullptr;
  moe::launch_add_norm(x, residual, norm_weight, eps, T, H, sum, norm, codes, scales, sms, s);
  moe::launch_router_chunked(norm, w_gate, router_bias, at<float>(ws, L.rpart), logits, nullptr, nullptr, T, H, N,
                             cfg->top_k, s);
  MOE_TRY(route_impl(cfg, scoring, T, logits, score_bias, idx, gates, s));
  moe::launch_dispatch(idx, T, N, cfg->top_k, cfg->block_size, api::capacity(cfg, T), kept, pos, sorted, blocks,
                       num_padded, at<int32_t>(ws, L.counts), at<int32_t>(ws, L.dropped), at<int32_t>(ws, L.rank),
                       at<int32_t>(ws, L.tile_count), at<int32_t>(ws, L.seg_off), at<int>(ws, L.status), s);
  MOE_TRY(ffn_impl(cfg, T, codes, scales, w, sorted, blocks, num_padded, y, y_sh, ws, s));
  moe::launch_combine(sum ? sum : x, gates, kept, pos, y, y_sh, out, T, H, cfg->top_k, api::max_rows(cfg, T), s);
  return api::last_error();
}

}  // extern "C"
