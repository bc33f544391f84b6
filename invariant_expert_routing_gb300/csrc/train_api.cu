// C ABI of the layer's training step (include/moe_api.h): products grouped by
// expert and their gradients, SwiGLU with gates, layer norm, the norms' gradients.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "api_internal.h"
#include "grouped.h"
#include "kernels.h"

namespace {

namespace api = moe::api;

constexpr int kMaxWidth = 65536;    // K, F
constexpr int kMaxHidden = 32768;   // H of the norms
constexpr size_t kGroupedWorkspace = 256;

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + bn && y < x + an;
}

// Whether an output lies over an input or over another output.  An input that an
// output may be in place of is left out (null) where it is that output.
struct Span {
  const void* p;
  size_t bytes;
};
bool clash(std::initializer_list<Span> out, std::initializer_list<Span> in) {
  for (const Span* o = out.begin(); o != out.end(); ++o) {
    for (const Span& i : in)
      if (overlap(o->p, o->bytes, i.p, i.bytes)) return true;
    for (const Span* q = o + 1; q != out.end(); ++q)
      if (overlap(o->p, o->bytes, q->p, q->bytes)) return true;
  }
  return false;
}
template <class T>
const T* unless(const void* same, const T* p) {
  return p == same ? nullptr : p;
}

moe_status check_width(int32_t n) {
  if (n <= 0) return MOE_ERR_INVALID_ARG;
  return n % 8 || n > kMaxWidth ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe_status check_norm(int32_t T, int32_t H, float eps) {
  if (T < 0 || H <= 0 || !(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
  return T > (1 << 20) || H % 8 || H > kMaxHidden ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

moe::GroupArgs group_args(const moe_config* c, int32_t T, int32_t K, int32_t F, const int32_t* ids,
                          const int32_t* counts, void* ws) {
  moe::GroupArgs g{};
  g.counts = counts;
  g.N = c->num_experts;
  g.B = c->block_size;
  g.max_rows = api::max_rows(c, T);
  g.ids = ids;
  g.T = T;
  g.slots = api::slots(c);
  g.K = K;
  g.F = F;
  g.status = static_cast<int*>(ws);
  g.wait_ns = (unsigned long long)c->debug_wait_ns;
  return g;
}

moe_status check_group(const moe_config* c, int32_t T, int32_t K, int32_t F) {
  MOE_TRY(api::check_config(c));
  MOE_TRY(api::check_tokens(c, T));
  MOE_TRY(check_width(K));
  return check_width(F);
}

}  // namespace

extern "C" {

size_t moe_workspace_bytes_grouped(const moe_config* cfg, int32_t max_tokens) {
  if (api::check_config(cfg) != MOE_OK || api::check_tokens(cfg, max_tokens) != MOE_OK) return 0;
  return kGroupedWorkspace;
}

moe_status moe_grouped_gemm(const moe_config* cfg, int32_t T, int32_t K, int32_t F, uint32_t flags, const uint16_t* x,
                            const uint16_t* w, const int32_t* sorted_route_ids, const int32_t* expert_counts,
                            uint16_t* y_perm, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_group(cfg, T, K, F));
  if (flags & ~(uint32_t)(MOE_GROUPED_GATHER | MOE_GROUPED_TRANSPOSED)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  const bool gather = flags & MOE_GROUPED_GATHER;
  MOE_TRY(api::need(x));
  MOE_TRY(api::need(w));
  MOE_TRY(gather ? api::need(sorted_route_ids) : api::optional(sorted_route_ids));
  MOE_TRY(api::need(expert_counts));
  MOE_TRY(api::need(y_perm));
  MOE_TRY(api::need(ws));
  if (ws_bytes < kGroupedWorkspace) return MOE_ERR_WORKSPACE;
  moe::GroupedGemmArgs a{};
  a.g = group_args(cfg, T, K, F, sorted_route_ids, expert_counts, ws);
  const size_t rows = (size_t)a.g.max_rows;
  if (clash({{y_perm, 2 * rows * F}, {ws, kGroupedWorkspace}},
            {{x, 2 * (gather ? (size_t)T : rows) * K},
             {w, 2 * (size_t)a.g.N * K * F},
             {gather ? sorted_route_ids : nullptr, sizeof(int32_t) * rows},
             {expert_counts, sizeof(int32_t) * (size_t)a.g.N}}))
    return MOE_ERR_INVALID_ARG;
  a.x = x;
  a.w = w;
  a.y = y_perm;
  a.gather = gather;
  a.transposed = (flags & MOE_GROUPED_TRANSPOSED) != 0;
  const int sms = api::sm_count();
  if (sms <= 0 || !moe::launch_grouped_gemm(a, api::tensor_map_encode(), sms, static_cast<cudaStream_t>(stream))) return MOE_ERR_CUDA;
  return api::last_error();
}

moe_status moe_grouped_wgrad(const moe_config* cfg, int32_t T, int32_t K, int32_t F, uint32_t flags, const uint16_t* x,
                             const uint16_t* dy, const int32_t* sorted_route_ids, const int32_t* expert_counts,
                             const float* dw_add, void* dw, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_group(cfg, T, K, F));
  if (flags & ~(uint32_t)(MOE_WGRAD_GATHER_X | MOE_WGRAD_GATHER_DY | MOE_WGRAD_BF16)) return MOE_ERR_INVALID_ARG;
  const bool bf16 = flags & MOE_WGRAD_BF16;
  if (bf16 && dw_add) return MOE_ERR_INVALID_ARG;
  MOE_TRY(api::need(dw));
  MOE_TRY(api::optional(dw_add));
  const size_t dw_bytes = (bf16 ? 2 : 4) * (size_t)cfg->num_experts * K * F;
  if (dw_add != dw && overlap(dw, dw_bytes, dw_add, dw_bytes)) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {   // a sum over no rows
    if (dw_add == dw) return MOE_OK;
    const cudaError_t e = dw_add ? cudaMemcpyAsync(dw, dw_add, dw_bytes, cudaMemcpyDeviceToDevice, s)
                                 : cudaMemsetAsync(dw, 0, dw_bytes, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  const bool gx = flags & MOE_WGRAD_GATHER_X, gd = flags & MOE_WGRAD_GATHER_DY;
  MOE_TRY(api::need(x));
  MOE_TRY(api::need(dy));
  MOE_TRY(gx || gd ? api::need(sorted_route_ids) : api::optional(sorted_route_ids));
  MOE_TRY(api::need(expert_counts));
  MOE_TRY(api::need(ws));
  if (ws_bytes < kGroupedWorkspace) return MOE_ERR_WORKSPACE;
  moe::GroupedWgradArgs a{};
  a.g = group_args(cfg, T, K, F, sorted_route_ids, expert_counts, ws);
  const size_t rows = (size_t)a.g.max_rows;
  if (clash({{dw, dw_bytes}, {ws, kGroupedWorkspace}},
            {{x, 2 * (gx ? (size_t)T : rows) * K},
             {dy, 2 * (gd ? (size_t)T : rows) * F},
             {unless(dw, dw_add), dw_bytes},
             {gx || gd ? sorted_route_ids : nullptr, sizeof(int32_t) * rows},
             {expert_counts, sizeof(int32_t) * (size_t)a.g.N}}))
    return MOE_ERR_INVALID_ARG;
  a.x = x;
  a.dy = dy;
  a.add = dw_add;
  a.dw = dw;
  a.gather_x = gx;
  a.gather_dy = gd;
  a.fp32 = !bf16;
  const int sms = api::sm_count();
  if (sms <= 0 || !moe::launch_grouped_wgrad(a, api::tensor_map_encode(), sms, s)) return MOE_ERR_CUDA;
  return api::last_error();
}

moe_status moe_swiglu(const moe_config* cfg, int32_t T, const uint16_t* gu, const float* topk_gate,
                      const int32_t* sorted_route_ids, const int32_t* num_padded, uint16_t* a, void* stream) {
  MOE_TRY(api::check_config(cfg));
  MOE_TRY(api::check_tokens(cfg, T));
  if (T == 0) return MOE_OK;
  MOE_TRY(api::need(gu));
  MOE_TRY(api::optional(topk_gate));
  MOE_TRY(api::need(sorted_route_ids));
  MOE_TRY(api::need(num_padded));
  MOE_TRY(api::need(a));
  const int64_t rows = api::max_rows(cfg, T);
  const int I = cfg->intermediate;
  const size_t gates = sizeof(float) * (size_t)T * api::slots(cfg);
  if (clash({{a, 2 * (size_t)rows * I}}, {{gu, 4 * (size_t)rows * I},
                                          {topk_gate, gates},
                                          {sorted_route_ids, sizeof(int32_t) * (size_t)rows},
                                          {num_padded, sizeof(int32_t)}}))
    return MOE_ERR_INVALID_ARG;
  moe::launch_swiglu(gu, topk_gate, sorted_route_ids, num_padded, rows, T * api::slots(cfg), I, a,
                     static_cast<cudaStream_t>(stream));
  return api::last_error();
}

moe_status moe_swiglu_backward(const moe_config* cfg, int32_t T, const uint16_t* gu, const float* topk_gate,
                               const uint16_t* da, const int32_t* sorted_route_ids, const int32_t* num_padded,
                               uint16_t* dgu, float* dgate, uint16_t* a, void* stream) {
  MOE_TRY(api::check_config(cfg));
  MOE_TRY(api::check_tokens(cfg, T));
  if (T == 0) return MOE_OK;
  MOE_TRY(api::need(gu));
  MOE_TRY(api::optional(topk_gate));
  MOE_TRY(api::need(da));
  MOE_TRY(api::need(sorted_route_ids));
  MOE_TRY(api::need(num_padded));
  MOE_TRY(api::need(dgu));
  MOE_TRY(api::optional(dgate));
  MOE_TRY(api::optional(a));
  const int64_t rows = api::max_rows(cfg, T);
  const int I = cfg->intermediate;
  const size_t one = 2 * (size_t)rows * I, gates = sizeof(float) * (size_t)T * api::slots(cfg);
  // (a CTA stores its row's entry of dgate while others still read gu and da)
  if (clash({{dgu, 2 * one}, {a, one}, {dgate, gates}}, {{unless(dgu, gu), 2 * one},
                                                         {unless(a, da), one},
                                                         {topk_gate, gates},
                                                         {sorted_route_ids, sizeof(int32_t) * (size_t)rows},
                                                         {num_padded, sizeof(int32_t)}}))
    return MOE_ERR_INVALID_ARG;
  moe::launch_swiglu_backward(gu, topk_gate, da, sorted_route_ids, num_padded, rows, T * api::slots(cfg), I, dgu, dgate,
                              a, static_cast<cudaStream_t>(stream));
  return api::last_error();
}

moe_status moe_add_layer_norm(int32_t T, int32_t H, const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                              const uint16_t* bias, float eps, uint16_t* residual_out, uint16_t* out, void* stream) {
  MOE_TRY(check_norm(T, H, eps));
  if (T == 0) return MOE_OK;
  MOE_TRY(api::need(x));
  MOE_TRY(api::optional(residual));
  MOE_TRY(api::need(weight));
  MOE_TRY(api::optional(bias));
  MOE_TRY(api::optional(residual_out));
  MOE_TRY(api::need(out));
  const size_t n = 2 * (size_t)T * H;
  for (const uint16_t* o : {(const uint16_t*)residual_out, (const uint16_t*)out})
    if (clash({{o, n}}, {{unless(o, x), n}, {unless(o, residual), n}, {weight, 2 * (size_t)H}, {bias, 2 * (size_t)H}}))
      return MOE_ERR_INVALID_ARG;
  if (overlap(out, n, residual_out, n)) return MOE_ERR_INVALID_ARG;
  const int sms = api::sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  moe::launch_add_layer_norm(x, residual, weight, bias, eps, T, H, residual_out, out, sms,
                             static_cast<cudaStream_t>(stream));
  return api::last_error();
}

size_t moe_workspace_bytes_norm_backward(int32_t max_tokens, int32_t H) {
  // (no tokens are as valid as any number, and need a workspace of no more than one)
  return check_norm(max_tokens, H, 0.0f) == MOE_OK ? moe::norm_backward_scratch_bytes(max_tokens ? max_tokens : 1, H) : 0;
}

moe_status moe_norm_backward(int32_t T, int32_t H, int32_t centre, const uint16_t* v, const uint16_t* dout,
                             const uint16_t* dresidual, const uint16_t* weight, float eps, uint16_t* dx, float* dweight,
                             float* dbias, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_norm(T, H, eps));
  if (centre != 0 && centre != 1) return MOE_ERR_INVALID_ARG;
  MOE_TRY(api::optional(dweight));
  MOE_TRY(api::optional(dbias));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {   // sums over no rows
    for (float* p : {dweight, dbias})
      if (p && cudaMemsetAsync(p, 0, sizeof(float) * H, s) != cudaSuccess) return MOE_ERR_CUDA;
    return MOE_OK;
  }
  MOE_TRY(api::need(v));
  MOE_TRY(api::need(dout));
  MOE_TRY(api::optional(dresidual));
  MOE_TRY(api::need(weight));
  MOE_TRY(api::need(dx));
  MOE_TRY(api::need(ws));
  const size_t scratch = moe::norm_backward_scratch_bytes(T, H);
  if (ws_bytes < scratch) return MOE_ERR_WORKSPACE;
  const size_t n = 2 * (size_t)T * H, sum_bytes = sizeof(float) * (size_t)H;
  // (the CTAs store their columns' sums into ws while others read rows and write dx)
  if (clash({{dx, n}, {dweight, sum_bytes}, {dbias, sum_bytes}, {ws, scratch}},
            {{v, n}, {dout, n}, {unless(dx, dresidual), n}, {weight, 2 * (size_t)H}}))
    return MOE_ERR_INVALID_ARG;
  moe::launch_norm_backward(v, dout, dresidual, weight, eps, T, H, centre != 0, dx, dweight, dbias, ws, s);
  return api::last_error();
}

}  // extern "C"
