/*
 * moe_api.h - C ABI of the batch-invariant Mixture-of-Experts layer forward
 * for NVIDIA GB300 (sm_103a).  Library: libmoe_gb300.so.
 *
 * The layer, per token h (row of h [T, H]):
 *   logits = h . W_g (+ bias)                          router, N scores
 *   experts, gates = top-k of softmax(logits), renormalised over the k
 *   capacity check per expert (overflowing routes are dropped)
 *   out = h + sum over kept routes of gate * SwiGLU_e(h)  (+ shared expert)
 * as stated in "Mixture-of-Experts Routing at Inference Time" (ACE Journal),
 * section "How sparse routing works", Figure 1, and "The hard part: token
 * dropping is a silent correctness bug", Figure 2; and in "Mixture-of-experts
 * routing and LLM repeatability" (the per-token pseudo-code, the Switch
 * capacity rule).  The split into route -> dispatch/align -> expert FFN ->
 * combine follows Figure 3 of the first page (router top-k, capacity check
 * and overflow policy, expert compute).
 *
 * Batch invariance ("Why temperature=0 Still Gives Different Answers: Batch
 * Invariance", section "What is batch invariance in LLM inference?"): every
 * reduction has one fixed split and order regardless of T, with no split-K
 * and no atomics, so a token's outputs are bitwise identical regardless of the
 * other tokens of the batch and whichever padded block its routes land in.  The only
 * exception is the capacity rule itself, which couples tokens by design.
 *
 * Conventions for every entry point:
 *   - Pointers are device memory owned by the caller unless the name says
 *     _host.  The library allocates no device memory; scratch comes from the
 *     caller's workspace `ws` of `ws_bytes` bytes (see moe_workspace_bytes).
 *   - bf16 tensors are passed as uint16_t bit patterns, row-major.
 *   - Every device pointer must be 16-byte aligned.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream).  Argument errors are returned synchronously before
 *     anything is launched.  MOE_ERR_CUDA reports a launch error.
 *   - T == 0 is a no-op that returns MOE_OK.
 *   - Device-side anomalies (an expert id outside [0, N) passed in through
 *     moe_dispatch_align, a pipeline wait that timed out) never trap: they set
 *     bits of the device status word held in the workspace, the offending work
 *     is skipped, and moe_get_device_status reports them.
 *   - Routes are numbered r = t*k + j (token t, slot j): the flattened route
 *     identifier of "Route-Block Membership Selects Packed-AWQ Arithmetic",
 *     section "The bookkeeping before the matrix multiplication".
 */
#ifndef MOE_API_H
#define MOE_API_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Overflow policy for routes past an expert's capacity ("Mixture-of-Experts
 * Routing at Inference Time", Figure 2): drop (the route adds nothing; the
 * token keeps its residual and its other routes) or reroute (the route moves
 * to the token's best-ranked expert that still has room and that the token
 * does not use yet; it keeps its slot's gate). */
#define MOE_OVERFLOW_DROP 0
#define MOE_OVERFLOW_REROUTE 1
/* Routing: token choice (each token takes its top-k experts) or expert choice
 * (each expert takes its top-C tokens of the batch by softmax probability;
 * "Mixture-of-experts routing and LLM repeatability"). */
#define MOE_ROUTING_TOKEN_CHOICE 0
#define MOE_ROUTING_EXPERT_CHOICE 1

/* Layer shape.  Supported: H % 128 == 0, I % 128 == 0, Is % 128 == 0,
 * 1 <= N <= 256, 1 <= k <= min(N, 16), B % 8 == 0 and 8 <= B <= 128 with
 * 128 % B == 0, T <= 1,048,576 and T*S < 2^31, S = route slots per token
 * (k for token choice, N for expert choice).  Zero-initialise the struct:
 * zero is the default of every field. */
typedef struct moe_config {
  int32_t hidden;              /* H */
  int32_t num_experts;         /* N routed experts */
  int32_t top_k;               /* k (expert choice: average experts per token) */
  int32_t intermediate;        /* I, routed expert FFN width */
  int32_t block_size;          /* B, rows per padded expert block */
  double capacity_factor;      /* > 0: capacity ceil(cf*T*k/N) per expert, in fp64 as
                                  ceil(((cf*T)*k)/N); <= 0: no limit (expert choice:
                                  cf = 1, capacity clipped to T) */
  int32_t shared_intermediate; /* Is of the always-on shared expert; 0: none */
  int32_t overflow_policy;     /* MOE_OVERFLOW_DROP or MOE_OVERFLOW_REROUTE (token choice) */
  int32_t routing;             /* MOE_ROUTING_TOKEN_CHOICE or MOE_ROUTING_EXPERT_CHOICE */
  /* Testing and diagnosis only; leave zero in production.  None of these
   * changes a result bit: each forces one of several equivalent ways of
   * computing the same integers and floats, or shortens the bounded waits. */
  uint32_t debug_flags;        /* MOE_DEBUG_* bits */
  int32_t debug_grid_ctas;     /* > 0: at most this many CTAs run the reroute's grid-wide
                                  rounds (more routes per CTA); 0: one per SM */
  int64_t debug_wait_ns;       /* > 0: every bounded device wait gives up after this many ns
                                  (the grouped GEMM's pipeline waits, default 2 s, and the
                                  reroute's grid barrier, default 0.2 s); 0: the defaults */
} moe_config;

/* debug_flags bits.  Each pair of alternatives computes the same bits; a
 * flag only selects which kernels run (the tests compare them). */
#define MOE_DEBUG_ROUTER_TC 0x1u          /* tensor-core router with the certified filter
                                             wherever it can serve the call (N % 128 == 0,
                                             no logits_out), whatever T */
#define MOE_DEBUG_ROUTER_CHUNKED 0x2u     /* chunked CUDA-core router for every batch */
#define MOE_DEBUG_ROW_GATHER 0x4u         /* routed token rows copied in segment order */
#define MOE_DEBUG_ROW_SCATTER 0x8u        /* routed token rows copied token by token
                                             (moe_forward; moe_expert_ffn always gathers) */
#define MOE_DEBUG_NO_DECODE_FRONT 0x10u   /* no fused decode front for T <= 2 */
#define MOE_DEBUG_REROUTE_SEQUENTIAL 0x20u /* reroute: the sequential kernel alone */
#define MOE_DEBUG_REROUTE_GRID 0x40u      /* reroute: grid-wide acceptance rounds for any batch */
#define MOE_DEBUG_REROUTE_ONE_CTA 0x80u   /* reroute: one-CTA acceptance rounds for any batch */
#define MOE_DEBUG_ROUTER_TILE128 0x100u   /* tensor-core router logits in 128-row token tiles */
#define MOE_DEBUG_ROUTER_TILE64 0x200u    /* tensor-core router logits in 64-row token tiles */
#define MOE_DEBUG_SHARED_SERIAL 0x400u    /* moe_forward: the shared expert on the caller's stream after
                                             the routed GEMMs instead of on a second stream */
#define MOE_DEBUG_W13_PAIR 0x800u         /* routed W13 on CTA pairs (the default wherever the
                                             intermediate size is a multiple of 128) */
#define MOE_DEBUG_W2_WIDE 0x1000u         /* routed W2 pairs in wide items (two 256-feature groups per
                                             token tile) whatever the reduction length */
#define MOE_DEBUG_W13_SINGLE 0x2000u      /* routed W13 on single CTAs (M = 128 features x N = 128
                                             token rows, gate and up MMAs per K step) */

/* Output of moe_routing_stats (device memory, 40 bytes). */
typedef struct moe_route_stats {
  int32_t max_expert_load;  /* routes naming the busiest expert */
  int32_t min_expert_load;  /* routes naming the idlest expert */
  int32_t capacity;         /* probe capacity floor(mean load * capacity_factor) */
  int32_t dropped_tokens;   /* sum over experts of max(0, load - capacity) */
  int32_t total_routes;     /* routes with an expert id in [0, N) */
  int32_t reserved;         /* 0 */
  double imbalance_ratio;   /* max load / mean load */
  double drop_fraction;     /* dropped_tokens / total_routes */
} moe_route_stats;

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1, /* null or misaligned pointer, negative size, inconsistent sizes */
  MOE_ERR_UNSUPPORTED = 2, /* shape outside the supported set above */
  MOE_ERR_WORKSPACE = 3,   /* workspace smaller than moe_workspace_bytes(cfg, T) */
  MOE_ERR_CUDA = 4,        /* a CUDA runtime/driver call failed */
  MOE_ERR_DEVICE = 5       /* the device status word has an error bit set */
} moe_status;

/* Bits of the device status word. */
#define MOE_DEV_ERR_EXPERT_RANGE 0x1 /* a topk_idx entry outside [0, N): route not dispatched */
#define MOE_DEV_ERR_TIMEOUT 0x2      /* a bounded pipeline wait gave up; outputs are invalid */
#define MOE_DEV_ERR_BAD_BLOCKS 0x4   /* moe_expert_ffn got a block list that is unsorted, out of
                                        range or longer than the bound: no expert work was done */
/* Informational bit (not an error; moe_get_device_status still returns
 * MOE_OK when it is the only bit set): the reroute's grid-wide acceptance
 * rounds gave up at a device-wide barrier that waited past its limit, and the
 * sequential kernel computed the assignment instead (valid results). */
#define MOE_DEV_NOTE_REROUTE_FALLBACK 0x100
#define MOE_DEV_ERR_MASK 0xFF        /* bits that mark invalid outputs */

/* Text for a status code (static storage). */
const char* moe_status_string(moe_status s);

/* Checks a configuration against the supported set. */
moe_status moe_check_config(const moe_config* cfg);

/* Expert capacity for a batch of T tokens: ceil(cf*T*k/N), or -1 (no limit).
 * Capacity per "Mixture-of-experts routing and LLM repeatability" (tokens per
 * expert times a capacity factor), rounded up.  Expert choice: the tokens
 * each expert takes, min(ceil(cf*T*k/N), T) with cf = 1 when cf <= 0. */
int32_t moe_capacity(const moe_config* cfg, int32_t T);

/* Upper bounds used to size caller buffers for T tokens:
 *   rows of sorted_route_ids (and of y_perm):  T*k + N*(B-1)
 *   entries of block_expert:                   (T*k)/B + N
 * Expert choice: N*P rows and N*P/B blocks exactly, P = moe_capacity rounded
 * up to a multiple of B. */
int64_t moe_max_padded_rows(const moe_config* cfg, int32_t T);
int64_t moe_max_blocks(const moe_config* cfg, int32_t T);

/* Bytes of workspace that every call below needs for up to max_tokens
 * tokens (0 if the configuration is invalid).  The workspace holds the
 * intermediate tensors of moe_forward, the tile list of the grouped GEMMs and
 * the device status word.  Contents need not be initialised; the layout is a
 * fixed function of (cfg, max_tokens), so a call with T <= max_tokens may use
 * any workspace sized for max_tokens. */
size_t moe_workspace_bytes(const moe_config* cfg, int32_t max_tokens);

/* Router: logits, softmax, top-k, renormalised gates ("Mixture-of-Experts
 * Routing at Inference Time", "How sparse routing works" and its TopKRouter).
 *   h        [T, H]  bf16        w_gate [H, N] bf16     router_bias [N] fp32 or NULL
 *   topk_idx [T, k]  int32 out   experts sorted by ascending index
 *   topk_gate[T, k]  fp32  out   exp(l_j - m) / sum_sel exp(l_s - m), m = max selected
 *   logits_out [T, N] fp32 out or NULL
 * Logits are fp32 with a fixed order: H cut into 256-element chunks, each
 * summed from +0 in ascending index, chunk sums added in ascending order to a
 * total starting at +0, bias added last (fixed-chunk reduction of "Why
 * temperature=0 Still Gives Different Answers", Tier 2).  Selection ranks
 * larger logits first, equal logits by lower expert index, NaN last. */
moe_status moe_route(const moe_config* cfg, int32_t T, const uint16_t* h, const uint16_t* w_gate,
                     const float* router_bias, int32_t* topk_idx, float* topk_gate,
                     float* logits_out, void* ws, size_t ws_bytes, void* stream);

/* The router logits alone: logits_out [T, N] fp32, every expert, in the
 * fixed order of moe_route (CUDA cores).  Input of expert-choice routing,
 * overflow reroute and the router margin. */
moe_status moe_router_logits(const moe_config* cfg, int32_t T, const uint16_t* h,
                             const uint16_t* w_gate, const float* router_bias, float* logits_out,
                             void* ws, size_t ws_bytes, void* stream);

/* Router paths.  With logits_out != NULL, when N is not a multiple of 128,
 * when H > 8192, for at most 64 tokens, or when T * H * N <= 3 * 2^28,
 * moe_route computes every logit in the canonical order on CUDA cores (the
 * chunked router: 256-element chunk sums in parallel CTAs, then an in-order
 * reduce with the top-k; two launches).
 * Otherwise (moe_forward, or moe_route without logits_out, N % 128 == 0) it
 * first computes l_tc = h . W_g on the tensor cores, bounds |l_tc - l| by
 * delta_t = beta(H) * ||h_t|| * max_e ||W_g[:,e]|| (+ bias rounding), keeps
 * as candidates the experts with l_tc >= L_k - 2 delta_t (L_k = k-th largest
 * l_tc; all experts if anything is non-finite) and computes canonical logits
 * for those only.  Experts below the cut provably cannot be in the top-k,
 * so topk_idx and topk_gate are bit-identical on both paths.
 *   beta(H) = (H/16 + 1) 2^-20 + (256 + ceil(H/256) + 1) 2^-24 covers
 *   H/16 tensor-core K=16 steps at a relative error of 2^-20 each (several
 *   times the truncation error of a 16-term fp32 block sum) and the fp32
 *   additions of the canonical order. */
float moe_router_cert_beta(int32_t hidden);

/* Diagnostic: the tensor-core logits l_tc = h . W_g [T, N] fp32 (no bias) that
 * the filter uses (MOE_ERR_UNSUPPORTED unless N % 128 == 0).  Not the
 * canonical logits; the router margin and the filter width can be studied
 * with them. */
moe_status moe_router_tc_logits(const moe_config* cfg, int32_t T, const uint16_t* h,
                                const uint16_t* w_gate, float* logits_out, void* ws,
                                size_t ws_bytes, void* stream);

/* Diagnostic: the tensor-core router path of moe_route (same topk_idx and
 * topk_gate), also reporting per token how many experts passed the filter
 * and had their canonical logits computed: n_candidates [T] int32 (k..N).
 * MOE_ERR_UNSUPPORTED unless N % 128 == 0 and H <= 8192. */
moe_status moe_route_filtered(const moe_config* cfg, int32_t T, const uint16_t* h,
                              const uint16_t* w_gate, const float* router_bias, int32_t* topk_idx,
                              float* topk_gate, int32_t* n_candidates, void* ws, size_t ws_bytes,
                              void* stream);

/* Capacity-limited dispatch and stable alignment into padded expert blocks.
 * Input topk_idx [T, k] (from moe_route, or recorded routes to replay).
 * Capacity is filled in batch order: an expert keeps its first C routes by
 * ascending route id; the rest are dropped and ride the residual (Figure 2 of
 * "Mixture-of-Experts Routing at Inference Time").  Stable construction
 * ("Route-Block Membership Selects Packed-AWQ Arithmetic", "Stable
 * construction selected a third trajectory"): for e = 0..N-1, expert e's kept
 * routes in ascending r, padded with the sentinel T*k to a multiple of B.
 * Outputs (device):
 *   route_kept      [T*k]                    uint8, 1 = kept
 *   route_pos       [T*k]                    int32, row in sorted_route_ids, -1 if not kept
 *   sorted_route_ids[moe_max_padded_rows]    int32, first *num_padded rows valid
 *   block_expert    [moe_max_blocks]         int32, first *num_padded/B valid
 *   num_padded      [1] int32,  expert_counts [N] int32 (kept), num_dropped [1] int32
 * Integer results only, no atomics: identical bits on every run. */
moe_status moe_dispatch_align(const moe_config* cfg, int32_t T, const int32_t* topk_idx,
                              uint8_t* route_kept, int32_t* route_pos, int32_t* sorted_route_ids,
                              int32_t* block_expert, int32_t* num_padded, int32_t* expert_counts,
                              int32_t* num_dropped, void* ws, size_t ws_bytes, void* stream);
/* One shard of a capacity-limited batch split across GPUs (or calls) in
 * token order: the same dispatch as moe_dispatch_align on the whole batch of
 * global_tokens tokens, restricted to this shard's routes.  The capacity is
 * C = moe_capacity(cfg, global_tokens); expert_offset [N] int32 (device; NULL
 * for the first shard) holds the routes each expert received in all earlier
 * shards (their moe_routing_stats expert_load, summed), so the shard's routes
 * to expert e keep what the earlier ones left: a route is kept iff its rank
 * among the shard's routes to e is below max(0, C - expert_offset[e]) — the
 * batch-order priority of the unsharded batch ("Mixture-of-Experts Routing
 * at Inference Time": capacity filled in batch order).  Obtaining
 * expert_offset takes one exchange of N integers per shard (an all-gather in
 * rank order); the layout, GEMMs and combine stay local.  Outputs as
 * moe_dispatch_align (this shard's routes and layout; num_dropped counts the
 * shard's dropped routes).  Drop policy and token choice only
 * (MOE_ERR_INVALID_ARG otherwise, or when global_tokens < T). */
moe_status moe_dispatch_align_shard(const moe_config* cfg, int32_t T, int32_t global_tokens,
                                    const int32_t* topk_idx, const int32_t* expert_offset,
                                    uint8_t* route_kept, int32_t* route_pos, int32_t* sorted_route_ids,
                                    int32_t* block_expert, int32_t* num_padded, int32_t* expert_counts,
                                    int32_t* num_dropped, void* ws, size_t ws_bytes, void* stream);

/* moe_dispatch_align implements the drop policy only: with
 * cfg->overflow_policy == MOE_OVERFLOW_REROUTE and a capacity in force, or with
 * expert-choice routing, it returns MOE_ERR_INVALID_ARG rather than dropping
 * routes the caller asked to keep (use the two entry points below). */

/* Capacity dispatch with the reroute overflow policy, then the same stable
 * alignment.  Phase one is moe_dispatch_align's capacity rule.  Phase two
 * takes the routes it would drop in ascending route id; each goes to the
 * best-ranked expert of its token (the router's order on logits [T, N], the
 * fp32 logits of every expert, e.g. from moe_router_logits) that has room left
 * and that the token does not use yet (its k chosen experts and the targets of
 * its earlier slots).  A route with no such expert is dropped.  The rerouted
 * route keeps its slot j and gate; moe_combine needs nothing else.
 * Outputs as moe_dispatch_align, plus
 *   route_expert [T*k] int32, expert each route is sent to, -1 if dropped
 *   num_rerouted [1] int32;  num_dropped counts the routes left dropped;
 *   expert_counts counts all routes each expert processes.
 * Integer results only: identical bits on every run.  cfg->overflow_policy is
 * not consulted (this entry point is the reroute policy). */
moe_status moe_dispatch_align_reroute(const moe_config* cfg, int32_t T, const int32_t* topk_idx,
                                      const float* logits, uint8_t* route_kept, int32_t* route_expert,
                                      int32_t* route_pos, int32_t* sorted_route_ids,
                                      int32_t* block_expert, int32_t* num_padded,
                                      int32_t* expert_counts, int32_t* num_dropped,
                                      int32_t* num_rerouted, void* ws, size_t ws_bytes, void* stream);

/* Expert-choice routing with its padded layout (cfg->routing must be
 * MOE_ROUTING_EXPERT_CHOICE).  From logits [T, N] (moe_router_logits) every
 * expert takes its C = moe_capacity(cfg, T) tokens of largest probability:
 * the key is log p = (l - m) - log(sum_e exp(l_e - m)) in fp64 (m = largest
 * logit, sum in ascending e; NaN logits rank last), equal keys by lower token
 * index.  A token may be taken by no expert (its output is then h plus the
 * shared expert).  Routes are r = t*N + e:
 *   gates       [T*N] fp32 out, softmax probability of every (t, e)
 *   route_kept  [T*N] uint8 out, 1 if expert e took token t
 *   route_pos   [T*N] int32 out, row in sorted_route_ids, -1 if not taken
 *   sorted_route_ids [moe_max_padded_rows], block_expert [moe_max_blocks],
 *   num_padded [1], expert_counts [N] (= C for every expert): as in
 *   moe_dispatch_align, expert e's tokens in ascending t, padded with T*N.
 * moe_expert_ffn and moe_combine then run with N slots per token. */
moe_status moe_route_expert_choice(const moe_config* cfg, int32_t T, const float* logits,
                                   float* gates, uint8_t* route_kept, int32_t* route_pos,
                                   int32_t* sorted_route_ids, int32_t* block_expert,
                                   int32_t* num_padded, int32_t* expert_counts, void* ws,
                                   size_t ws_bytes, void* stream);

/* The routing_stats probe of "Mixture-of-Experts Routing at Inference Time"
 * (section "The hard part: token dropping is a silent correctness bug") on
 * topk_idx [T, k] (token choice): expert_load [N] int32 out (routes naming
 * each expert), stats (device) out.  capacity_factor sets the probe's own
 * capacity floor(mean * cf) (1.25 in the page's probe); it is independent of
 * the layer's capacity.  fp64 results are single IEEE operations on the
 * integer counts.  Asynchronous; ids outside [0, N) are not counted. */
moe_status moe_routing_stats(const moe_config* cfg, int32_t T, const int32_t* topk_idx,
                             double capacity_factor, int32_t* expert_load, moe_route_stats* stats,
                             void* stream);

/* Router margin per token ("Mixture-of-experts routing and LLM
 * repeatability"): margin [T] fp64 out = l_(k) - l_(k+1), the k-th and
 * (k+1)-th logits of logits [T, N] under the router's ranking, as the fp64
 * difference of the two fp32 values; +inf when k = N, NaN if either is NaN.
 * A small margin marks a token whose experts a small numerical change can
 * flip. */
moe_status moe_router_margin(const moe_config* cfg, int32_t T, const float* logits, double* margin,
                             void* stream);

/* Grouped SwiGLU expert FFN over the padded blocks, on tcgen05 tensor cores:
 *   for every padded row p of expert e = block_expert[p / B] with route r:
 *     x = h[r / S] (S = k, or N for expert choice; zero for the sentinel),
 *     [g | u] = x . W13_e,
 *     a = bf16(silu(g) * u), y_perm[p] = bf16(a . W2_e)  (fp32 accumulation)
 *   and, when cfg->shared_intermediate > 0, y_shared[t] = SwiGLU_shared(h[t]).
 *   w13 [N, H, 2I] bf16 (gate columns 0..I-1, up columns I..2I-1),
 *   w2 [N, I, H] bf16, w13_shared [H, 2Is], w2_shared [Is, H] (or NULL when
 *   Is == 0); y_perm [moe_max_padded_rows, H] bf16 out; y_shared [T, H] bf16
 *   out or NULL when Is == 0 (the expert outputs are stored in bf16: half the
 *   bytes of the W2 store and of the combine's reads; every sum stays fp32).
 *   Rows of y_perm past the last route of an expert's segment (its padding),
 *   and past *num_padded, are not written.  A list of the caller's own may
 *   hold the sentinel or another id outside [0, T*S) before that route: such
 *   a row is computed from a row of zeros and written (zero for finite weights).
 * One tile shape and one K order for every T, no split-K: each y row
 * depends only on its own x row and the expert's weights. */
moe_status moe_expert_ffn(const moe_config* cfg, int32_t T, const uint16_t* h, const uint16_t* w13,
                          const uint16_t* w2, const uint16_t* w13_shared,
                          const uint16_t* w2_shared, const int32_t* sorted_route_ids,
                          const int32_t* block_expert, const int32_t* num_padded, uint16_t* y_perm,
                          uint16_t* y_shared, void* ws, size_t ws_bytes, void* stream);

/* Gate-weighted combine into the residual:
 *   out[t] = bf16( h[t] + sum_{j ascending, kept} topk_gate[t,j] * y_perm[route_pos[t*S+j]]
 *                  + y_shared[t] )
 * accumulated in fp32 in that fixed order (y_perm, y_shared bf16 as written
 * by moe_expert_ffn); S = k slots per token (N for expert choice, whose
 * gates are the [T, N] probabilities).  y_shared may be NULL.  out [T,H]
 * bf16. */
moe_status moe_combine(const moe_config* cfg, int32_t T, const uint16_t* h, const float* topk_gate,
                       const uint8_t* route_kept, const int32_t* route_pos, const uint16_t* y_perm,
                       const uint16_t* y_shared, uint16_t* out, void* stream);

/* The whole layer: moe_route -> moe_dispatch_align -> moe_expert_ffn ->
 * moe_combine on `stream`, intermediates in the workspace.  No host
 * synchronisation and no device-to-host copy.  With the reroute policy (and
 * a capacity) the router computes every logit canonically and the dispatch is
 * moe_dispatch_align_reroute; with expert-choice routing it is
 * moe_router_logits -> moe_route_expert_choice -> moe_expert_ffn ->
 * moe_combine. */
moe_status moe_forward(const moe_config* cfg, int32_t T, const uint16_t* h, const uint16_t* w_gate,
                       const float* router_bias, const uint16_t* w13, const uint16_t* w2,
                       const uint16_t* w13_shared, const uint16_t* w2_shared, uint16_t* out,
                       void* ws, size_t ws_bytes, void* stream);

/* moe_forward with the token rows in host memory: copies h_host [T, H] to the
 * device (into the workspace), runs the layer and copies the result back to
 * out_host [T, H].  Weights stay on the device.  Host buffers should be
 * page-locked for the copies to be asynchronous; the call returns after
 * enqueueing and the caller synchronises `stream` before reading out_host. */
moe_status moe_forward_hostio(const moe_config* cfg, int32_t T, const uint16_t* h_host,
                              const uint16_t* w_gate, const float* router_bias,
                              const uint16_t* w13, const uint16_t* w2,
                              const uint16_t* w13_shared, const uint16_t* w2_shared,
                              uint16_t* out_host, void* ws, size_t ws_bytes, void* stream);

/* moe_forward that also records caller-created CUDA events (cudaEvent_t
 * handles, at least n_events = 8) on `stream` at the stage boundaries:
 *   events[0] before the router          events[4] after the W13 GEMM
 *   events[1] after the router           events[5] after the W2 GEMM
 *   events[2] after dispatch/alignment   events[6] after the shared expert
 *   events[3] after tile list + row gather   events[7] after the combine
 * so the caller can read per-kernel device times (cudaEventElapsedTime)
 * without extra synchronisation.  Same computation and bits as moe_forward. */
moe_status moe_forward_timed(const moe_config* cfg, int32_t T, const uint16_t* h,
                             const uint16_t* w_gate, const float* router_bias, const uint16_t* w13,
                             const uint16_t* w2, const uint16_t* w13_shared,
                             const uint16_t* w2_shared, uint16_t* out, void* ws, size_t ws_bytes,
                             void* const* events, int32_t n_events, void* stream);

/* Number of kernel launches one moe_forward of T tokens makes for this
 * configuration (the router takes two on CUDA cores or six on the tensor
 * cores; at most 1024 routes are dispatched and cut into both GEMM tile lists
 * in one launch; for at most two tokens the router's chunk sums are followed
 * by one launch that routes, dispatches and gathers the routed rows, so a
 * forward without a shared expert is five launches). */
int32_t moe_forward_launch_count(const moe_config* cfg, int32_t T);

/* moe_dispatch_align for callers that cannot allocate device memory (for
 * example a serving loop whose memory is fixed at start-up, or code running
 * while another framework owns the allocator), so cannot pass a workspace.
 * The pages have no counterpart to this entry point; it is a deployment aid.
 * Same inputs, outputs and bits as moe_dispatch_align, but it allocates
 * nothing: its scratch is one fixed device array inside this library
 * (~321 KB on every GPU that loads it, held until the process exits).
 *   - Limit: T*k <= 65536 routes (and N <= 256); larger batches return
 *     MOE_ERR_UNSUPPORTED without doing anything.
 *   - status_out: device int32 or NULL; receives this call's device status
 *     word (MOE_DEV_ERR_EXPERT_RANGE for expert ids outside [0, N)).
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture.  A new context on the device (after
 *     cudaDeviceReset, for example) moves the array: the next call notices
 *     the change of context and looks the address up again, so make the
 *     first call after a reset before any capture too.
 *   - Every call on a device shares the one array, which keeps the previous
 *     call's contents (the call clears what must start at zero).  Calls that
 *     overlap on the GPU (e.g. on two streams at once) race on it: order them. */
moe_status moe_dispatch_align_noalloc(const moe_config* cfg, int32_t T, const int32_t* topk_idx,
                                      uint8_t* route_kept, int32_t* route_pos,
                                      int32_t* sorted_route_ids, int32_t* block_expert,
                                      int32_t* num_padded, int32_t* expert_counts,
                                      int32_t* num_dropped, int32_t* status_out, void* stream);

/* ------------------------------------------------------------------------
 * The layer on 4-bit experts: residual + RMS norm, routing by scores,
 * microscaled (MX) 4-bit tensors and the grouped expert FFN on them.
 *
 * An MX tensor [rows, K] (K % 32 == 0) is two byte arrays, row-major:
 *   codes  [rows, K/2]   two e2m1 values a byte, the even element in the low
 *                        half; sign, 2 exponent bits, 1 mantissa bit:
 *                        0, 0.5, 1, 1.5, 2, 3, 4, 6
 *   scales [rows, K/32]  one E8M0 byte b per 32 elements: 2^(b - 127); 255: NaN
 * A block of 32 converts with the exponent floor(log2(amax)) - 2 of its
 * largest magnitude amax (at least -127, which an all-zero block takes); each
 * element is rounded to the nearest value, ties to the even mantissa, and
 * saturates at 6.  A block that holds an infinity or a NaN gets the scale 255
 * and zero codes: all its elements read as NaN.
 * ------------------------------------------------------------------------ */

/* Residual addition, root-mean-square norm and the normalised row in 4 bits:
 *   v = x + residual (fp32);  residual_out = bf16(v)
 *   out = bf16(v / sqrt(mean(v^2) + eps) * weight)
 *   codes, scales = the MX tensor of out (the bf16 values, stored or not)
 *   x, residual [T, H] bf16 (residual NULL: v = x), weight [H] bf16,
 *   residual_out [T, H] bf16 or NULL, out [T, H] bf16 or NULL,
 *   codes [T, H/2] and scales [T, H/32], both or neither; out or codes given.
 * residual_out may be x or residual itself (each row is read before it is
 * written), and so may out; no other overlap.  H % 32 == 0, H <= 32768.  The sum of squares
 * has one order for every T.  It is fp32: with values past 1.8e19 it is infinite
 * (out is 0), and with eps = 0 it may vanish (values below about 1e-23: out is
 * infinite, and NaN where v is 0). */
moe_status moe_add_norm(int32_t T, int32_t H, const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                        float eps, uint16_t* residual_out, uint16_t* out, uint8_t* codes, uint8_t* scales,
                        void* stream);

/* How moe_route_scored scores and selects.  Zero-initialise: zero is the
 * default of every field. */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
#define MOE_GROUP_MAX 0
#define MOE_GROUP_TOP2_SUM 1
typedef struct moe_scoring {
  int32_t score;        /* MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID */
  int32_t num_groups;   /* groups of N / num_groups consecutive experts; 0, 1: no groups; <= 32 */
  int32_t top_groups;   /* groups a token may use; 0: all */
  int32_t group_score;  /* MOE_GROUP_MAX or MOE_GROUP_TOP2_SUM (groups of at least two) */
  int32_t renormalize;  /* 1: gates divided by the sum of the selected scores */
  float scale;          /* factor of the gates; 0: 1 */
} moe_scoring;

/* Checks a scoring against a configuration (token choice; top_k experts have
 * to fit into top_groups groups). */
moe_status moe_check_scoring(const moe_config* cfg, const moe_scoring* scoring);

/* Top-k routing by scores, from the logits of every expert (e.g. of
 * moe_router_logits):
 *   s = softmax(l) or 1 / (1 + exp(-l));  b = s + score_bias (selection only)
 *   groups rank by the largest b or the sum of the two largest; the experts
 *   outside the top_groups best are left out (not scored as zero)
 *   the k largest b; gate = scale * s, with renormalize scale * s / (sum of the
 *   selected s + 1e-20), the sum in one order for every T
 *   logits [T, N] fp32, score_bias [N] fp32 or NULL
 *   topk_idx [T, k] int32 out, experts in ascending index; topk_gate [T, k] fp32 out
 * Ties go to the lower index (of expert and of group); NaN ranks last.  A row
 * of -inf logits has softmax scores of zero.  Scores are fp32: sigmoid is 0 below
 * l = -88.7, softmax 0 some 104 below the largest logit, and what ranks is b, not
 * l.  moe_route ranks by the logits, so the two may choose differently where
 * unequal logits have equal scores. */
moe_status moe_route_scored(const moe_config* cfg, const moe_scoring* scoring, int32_t T, const float* logits,
                            const float* score_bias, int32_t* topk_idx, float* topk_gate, void* stream);

/* x [rows, K] bf16 -> MX tensor. */
moe_status moe_quantize_mx(int64_t rows, int32_t K, const uint16_t* x, uint8_t* codes, uint8_t* scales,
                           void* stream);
/* MX tensor -> out [rows, K] bf16 (exact, but for values past bf16's range). */
moe_status moe_dequantize_mx(int64_t rows, int32_t K, const uint8_t* codes, const uint8_t* scales, uint16_t* out,
                             void* stream);
/* Expert weights as moe_expert_ffn takes them, w [experts, K, F] bf16, to the
 * K-major MX tensor [experts, F, K] (blocks along K): w13 [N, H, 2I] -> [N,
 * 2I, H], w2 [N, I, H] -> [N, H, I].  K % 32 == 0, F % 8 == 0. */
moe_status moe_quantize_weights_mx(int32_t experts, int32_t K, int32_t F, const uint16_t* w, uint8_t* codes,
                                   uint8_t* scales, void* stream);
/* Scales of an MX weight tensor [experts, rows, K/32] in the order the GEMMs
 * read them (same number of bytes; done once, when the weights are loaded).
 * gate_up = 1 for w13 and w13_shared, 0 for w2 and w2_shared.  rows % 128 ==
 * 0, K % 128 == 0; scales and packed may not overlap (MOE_ERR_INVALID_ARG). */
moe_status moe_pack_scales_mx(int32_t experts, int32_t rows, int32_t K, int32_t gate_up, const uint8_t* scales,
                              uint8_t* packed, void* stream);

/* Bytes of workspace of moe_expert_ffn_mx and moe_forward_mx for up to
 * max_tokens tokens (0 if the configuration is invalid).  The device status
 * word is at its start, as in moe_workspace_bytes. */
size_t moe_workspace_bytes_mx(const moe_config* cfg, int32_t max_tokens);

/* moe_expert_ffn on 4-bit operands: for every padded row p with route r of
 * expert e,
 *   [g | u] = x[r / S] . W13_e,  a = MX(silu(g) * u),  y_perm[p] = bf16(a . W2_e)
 * x, W and a MX tensors, fp32 accumulation, silu(g) * u rounded once (fp32 to
 * e2m1).  With shared_intermediate > 0 y_shared[t] is the shared expert's
 * output.
 *   x_codes [T, H/2], x_scales [T, H/32]
 *   w13 [N, 2I, H/2] (gate rows 0..I-1, up rows I..2I-1), w2 [N, H, I/2], and
 *   w13_shared [2Is, H/2], w2_shared [H, Is/2] (or NULL): codes; their scales
 *   as moe_pack_scales_mx writes them
 *   sorted_route_ids, block_expert, num_padded, y_perm, y_shared: as in moe_expert_ffn
 *   (also which rows of y_perm are written)
 * One K order and no split-K: a row does not depend on the batch. */
moe_status moe_expert_ffn_mx(const moe_config* cfg, int32_t T, const uint8_t* x_codes, const uint8_t* x_scales,
                             const uint8_t* w13, const uint8_t* w13_scales, const uint8_t* w2,
                             const uint8_t* w2_scales, const uint8_t* w13_shared, const uint8_t* w13_shared_scales,
                             const uint8_t* w2_shared, const uint8_t* w2_shared_scales,
                             const int32_t* sorted_route_ids, const int32_t* block_expert, const int32_t* num_padded,
                             uint16_t* y_perm, uint16_t* y_shared, void* ws, size_t ws_bytes, void* stream);

/* Diagnostic: token rows of a tile of moe_expert_ffn_mx's routed experts, 32, 128
 * or 256, which follow the rows that an expert averages (T*k / N; with expert
 * choice moe_capacity): no result bit depends on it.  0 if the configuration is
 * invalid. */
int32_t moe_expert_ffn_mx_tile_rows(const moe_config* cfg, int32_t T);

/* A pre-norm MoE layer on 4-bit experts:
 *   v, n, MX(n) = moe_add_norm(x, residual);  logits = moe_router_logits(n)
 *   moe_route_scored -> moe_dispatch_align -> moe_expert_ffn_mx(MX(n))
 *   out = moe_combine with h = bf16(v): v + sum of gate * y + y_shared
 * residual NULL: v = x.  Token choice; the drop policy where a capacity is
 * set.  Weights as in moe_expert_ffn_mx, w_gate and router_bias as in
 * moe_route, score_bias as in moe_route_scored; out [T, H] bf16. */
moe_status moe_forward_mx(const moe_config* cfg, const moe_scoring* scoring, int32_t T, const uint16_t* x,
                          const uint16_t* residual, const uint16_t* norm_weight, float eps, const uint16_t* w_gate,
                          const float* router_bias, const float* score_bias, const uint8_t* w13,
                          const uint8_t* w13_scales, const uint8_t* w2, const uint8_t* w2_scales,
                          const uint8_t* w13_shared, const uint8_t* w13_shared_scales, const uint8_t* w2_shared,
                          const uint8_t* w2_shared_scales, uint16_t* out, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * The layer's training step on bf16 experts: the products grouped by expert
 * with the gradients of their inputs and weights, SwiGLU with the gates and
 * its gradient, layer norm, and the gradients of both norms.
 *
 * A forward that keeps what the gradient needs, and its gradient (S = slots
 * per token, H -> 2I -> H; ids and counts from moe_dispatch_align or
 * moe_route_expert_choice):
 *   gu    = moe_grouped_gemm(h, w13, GATHER)              [rows, 2I]
 *   a     = moe_swiglu(gu, gates)                         [rows, I]
 *   y     = moe_grouped_gemm(a, w2)                       [rows, H]
 *   out   = moe_combine(h, gates of 1, y)
 *   dw2   = moe_grouped_wgrad(a, dout, GATHER_DY)
 *   da    = moe_grouped_gemm(dout, w2, GATHER | TRANSPOSED)
 *   dgu, dgate = moe_swiglu_backward(gu, gates, da)
 *   dw13  = moe_grouped_wgrad(h, dgu, GATHER_X)
 *   dx    = moe_grouped_gemm(dgu, w13, TRANSPOSED)        [rows, H]
 *   dh    = moe_combine(dout, gates of 1, dx)
 * The step starts and ends at the gates: the gradient from dgate through the
 * (renormalised) scores into w_gate, the router's bias and the layer's input is
 * the caller's to compute and to add to dh, and so is a shared expert's.
 *
 * Rows are grouped as the dispatch lays them out: expert e's segment starts
 * at the sum of the earlier experts' expert_counts, each rounded up to a
 * multiple of B, and holds expert_counts[e] rows.  A gathered operand is
 * [T, columns]: row p of the segment reads its row sorted_route_ids[p] / S (an
 * id outside [0, T*S) reads zeros).  An operand in place is [rows, columns],
 * rows = moe_max_padded_rows(cfg, T).  Rows of the padding are not written
 * and change no result, whatever they hold (a product in place may load them with
 * the rows before them).  Counts that are negative or need more than
 * rows rows set MOE_DEV_ERR_BAD_BLOCKS and nothing is computed.
 * cfg gives N, B, the slots and the bound on the rows; K and F are multiples
 * of 8 up to 65536, free of cfg's hidden and intermediate.
 * ------------------------------------------------------------------------ */

/* Bytes of workspace of moe_grouped_gemm and moe_grouped_wgrad for up to
 * max_tokens tokens (0 if the configuration is invalid): the device status
 * word at its start, nothing kept from call to call (calls in flight at once
 * may share it). */
size_t moe_workspace_bytes_grouped(const moe_config* cfg, int32_t max_tokens);

/* y_perm[p] = bf16(x[row(p)] . W_e), fp32 accumulation, for every row p of
 * every expert e's segment.
 *   x [T, K] (GATHER) or [rows, K] bf16;  y_perm [rows, F] bf16 out
 *   w [N, K, F] bf16, with TRANSPOSED [N, F, K] (the product with W_e^T: the
 *   gradient of the input of a product with w [N, F, K])
 * sorted_route_ids may be NULL without GATHER.  y_perm and ws overlap nothing
 * else that the call is given.  One K order for every T, no split-K: a row does not
 * depend on the batch.  The tensor cores add 16 products of K at a time and
 * truncate the sum to fp32: off by at most K / 16 steps of 2^-23 of the sum so
 * far, before the one rounding to bf16 (2^-8 of the result). */
#define MOE_GROUPED_GATHER 0x1u
#define MOE_GROUPED_TRANSPOSED 0x2u
moe_status moe_grouped_gemm(const moe_config* cfg, int32_t T, int32_t K, int32_t F, uint32_t flags, const uint16_t* x,
                            const uint16_t* w, const int32_t* sorted_route_ids, const int32_t* expert_counts,
                            uint16_t* y_perm, void* ws, size_t ws_bytes, void* stream);

/* dw[e] = dw_add[e] + sum over the rows p of expert e's segment of
 * x[row(p)]^T dy[row(p)], in ascending p (fp32 accumulation, no atomics: the
 * same bits on every run).  An expert without rows gets dw_add or zeros.
 *   x  [T, K] (GATHER_X) or [rows, K] bf16, dy [T, F] (GATHER_DY) or [rows, F]
 *   dw [N, K, F] fp32 out, with BF16 bf16 (rounded once)
 *   dw_add [N, K, F] fp32 or NULL, may be dw itself (no other overlap of dw or
 *   ws with what the call is given); not with BF16
 * T = 0 writes dw too: dw_add or zeros. */
#define MOE_WGRAD_GATHER_X 0x1u
#define MOE_WGRAD_GATHER_DY 0x2u
#define MOE_WGRAD_BF16 0x4u
moe_status moe_grouped_wgrad(const moe_config* cfg, int32_t T, int32_t K, int32_t F, uint32_t flags, const uint16_t* x,
                             const uint16_t* dy, const int32_t* sorted_route_ids, const int32_t* expert_counts,
                             const float* dw_add, void* dw, void* ws, size_t ws_bytes, void* stream);

/* a[p] = bf16(w silu(g) u) for every row p < *num_padded whose route
 * r = sorted_route_ids[p] is in [0, T*S): g, u the halves of gu[p], silu(g) =
 * g / (1 + e^-g), w = topk_gate[r] (1 if topk_gate is NULL).  Other rows of a
 * are not written.
 *   gu [rows, 2I] bf16 (I = cfg->intermediate; the output of moe_grouped_gemm
 *   with w13), topk_gate [T, S] fp32 or NULL, a [rows, I] bf16 out, no overlap.
 * 1 / (1 + e^-g) is formed with the hardware's exponential and division, off by at
 * most (6 + 1.2 |g|) 2^-23 of it for g >= -87.3; below, where silu(g) is less than
 * 2^-119, it is 0 instead.
 * With the gate here the second product needs none: moe_combine then runs
 * with gates of 1. */
moe_status moe_swiglu(const moe_config* cfg, int32_t T, const uint16_t* gu, const float* topk_gate,
                      const int32_t* sorted_route_ids, const int32_t* num_padded, uint16_t* a, void* stream);

/* The gradient of moe_swiglu: with s = 1 / (1 + e^-g), per row
 *   dgu = bf16[ w da u s (1 + g (1 - s)) | w da silu(g) ]
 *   dgate[r] = sum over I of da silu(g) u   (fp32, one order for every T; each
 *   silu(g) as far off as in moe_swiglu)
 *   a as in moe_swiglu (the activation need not be kept for the weight gradient)
 *   da [rows, I] bf16, dgu [rows, 2I] bf16 out, dgate [T, S] fp32 out or NULL
 *   (entries of routes that are in no row are not written), a [rows, I] bf16
 *   out or NULL.
 * dgu may be gu and a may be da; no other overlap. */
moe_status moe_swiglu_backward(const moe_config* cfg, int32_t T, const uint16_t* gu, const float* topk_gate,
                               const uint16_t* da, const int32_t* sorted_route_ids, const int32_t* num_padded,
                               uint16_t* dgu, float* dgate, uint16_t* a, void* stream);

/* Residual addition and layer norm:
 *   v = x + residual (fp32);  residual_out = bf16(v)
 *   out = bf16((v - mean(v)) / sqrt(var(v) + eps) * weight + bias)
 *   x, residual [T, H] bf16 (residual NULL: v = x), weight [H] bf16, bias [H]
 *   bf16 or NULL, residual_out [T, H] bf16 or NULL, out [T, H] bf16.
 * var is the mean square of the deviations from the mean, computed from them.
 * residual_out may be x or residual itself, and so may out; no other overlap.
 * H % 8 == 0, H <= 32768.  Sums are fp32 in one order for every T.  With eps = 0
 * a row of equal values has no norm: NaN where the sum of its values is exact,
 * otherwise what the mean's rounding leaves. */
moe_status moe_add_layer_norm(int32_t T, int32_t H, const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                              const uint16_t* bias, float eps, uint16_t* residual_out, uint16_t* out, void* stream);

/* Bytes of workspace of moe_norm_backward for up to max_tokens rows (0 if
 * max_tokens or H is invalid).  Calls in flight at once need one each. */
size_t moe_workspace_bytes_norm_backward(int32_t max_tokens, int32_t H);

/* The gradient of moe_add_layer_norm (centre = 1) or moe_add_norm (centre =
 * 0) with respect to v and the parameters:
 *   n = (v - mean) / root, root = sqrt(var + eps) (RMS norm: mean = 0, var =
 *   mean(v^2)); g = dout * weight
 *   dx = bf16(dresidual + (g - mean(g) - n mean(g n)) / root)  (RMS norm
 *   without mean(g)): the gradient of x and of residual
 *   dweight = sum over t of dout n;  dbias = sum over t of dout
 *   v [T, H] bf16 (the forward's residual_out, or x without a residual), dout
 *   [T, H] bf16, dresidual [T, H] bf16 or NULL (the gradient of residual_out),
 *   weight [H] bf16, dx [T, H] bf16 out, dweight, dbias [H] fp32 out or NULL.
 * The statistics are computed again from v.  dx may be dresidual; no other
 * overlap.  The sums over rows have one order for a given T and H, without
 * atomics.  T = 0 sets dweight and dbias to zero.  H as above.
 * moe_add_layer_norm and moe_add_norm normalise x + residual in fp32; this takes
 * the statistics and n from v, which was rounded: in a row whose mean is m
 * deviations n is up to about m 2^-8 off.  With eps = 0 one row without deviation
 * makes all of dweight NaN, beside its row of dx. */
moe_status moe_norm_backward(int32_t T, int32_t H, int32_t centre, const uint16_t* v, const uint16_t* dout,
                             const uint16_t* dresidual, const uint16_t* weight, float eps, uint16_t* dx, float* dweight,
                             float* dbias, void* ws, size_t ws_bytes, void* stream);

/* Reads the device status word of `ws` (synchronises `stream`): the whole word
 * in *status_out; MOE_ERR_DEVICE if any bit of MOE_DEV_ERR_MASK is set. */
moe_status moe_get_device_status(const void* ws, int32_t* status_out, void* stream);

/* Clears the device status word of `ws` (asynchronous on `stream`). */
moe_status moe_clear_device_status(void* ws, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_API_H */
