/*
 * epx: MoE expert-parallel token dispatch and combine for one GPU's share of
 * the work, on AMD Instinct MI355X (gfx950).
 *
 * Destination ranks are modelled as segments of one receive buffer in HBM:
 * segment s holds the rows for experts [s*E/S, (s+1)*E/S).  Nothing here
 * moves data between GPUs.
 *
 * Conventions for every call below:
 *  - All buffers are caller-owned device memory (e.g. torch tensors).  The
 *    library never allocates, frees or synchronizes; every call enqueues its
 *    kernels on `stream` (a hipStream_t, NULL = the null stream) and returns.
 *  - Calls are stateless and reentrant.  Two calls that share an output
 *    buffer or a workspace must be ordered by the caller (same stream).
 *  - bf16 values travel as uint16_t bit patterns; float is IEEE binary32.
 *  - Payload pointers (x, recv, expert_out, y, grads, codes) must be 16-byte
 *    aligned; index buffers 4-byte aligned.
 *  - Return value: EP_OK, or a negative status (see ep_strerror).  Argument
 *    errors are found on the host before anything is enqueued.  Data errors
 *    (dropped slots, ids out of range) are reported on the device, in the
 *    layout's flags word, and never make a call fail.
 *
 * Sources for the semantics (page title, API item):
 *  [FA] NeMo AutoModel fused_a2a page: HybridEPDispatch.forward (tokens
 *       [tokens, hidden] -> [dispatched_tokens, hidden] grouped by local
 *       expert; topk_idx with -1 for unused slots; pad_multiple;
 *       num_permuted_tokens as a static, host-known output extent),
 *       HybridEPDispatch.backward (combine the gradients),
 *       HybridEPCombine.forward / backward (restore token order;
 *       redispatch the gradients).
 *  [TD] NeMo AutoModel token_dispatcher page: _align_up,
 *       TokenDispatcherConfig.moe_router_expert_pad_multiple,
 *       TokenDispatcherConfig.moe_router_dtype (fp32 weighted averaging),
 *       _assert_no_hybridep_overflow (device overflow flag, truncation at
 *       capacity), _HybridEPManager._calibrate_hybridep_capacity,
 *       _DeepepManager reversed_mapping_for_combine.
 *  [MX] MAX DistributedEPDispatchBlockScaledNVDynGlobalScales page, execute:
 *       NVFP4 with a per-token global scale 2688/rowmax, output_scales,
 *       output_rowwise_scales (BF16 inverse global scale), row_offsets,
 *       scales_offsets, expert_ids, src_info, atomic_counters,
 *       fused_shared_expert.
 */
#ifndef EPX_H
#define EPX_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define EPX_ABI_VERSION 1

/* Status codes. */
#define EP_OK 0
#define EP_EINVAL (-1)   /* an argument fails a host-side check                */
#define EP_ELAUNCH (-2)  /* the HIP runtime reported an error enqueueing work  */
#define EP_ENOTSUP (-3)  /* the current device is not gfx950                   */
#define EP_ESCRATCH (-4) /* ep_dispatch_layout_noalloc: the layout needs more
                            scratch than EP_NOALLOC_SCRATCH_BYTES             */
/* A HIP grid dimension holds at most 2^32 - 1 work-items.  ep_dispatch,
 * ep_combine, ep_dispatch_bwd and ep_combine_bwd split larger batches into
 * several launches.  The calls that launch one grid per batch return
 * EP_EINVAL past it: ep_dispatch_nvfp4, ep_dispatch_fp8 and the routing-map
 * conversions from T = 2^26 - 16 tokens (one wave per token), and
 * ep_combine_bwd_probs from T = 2^24 - 4 (one 256-thread workgroup per
 * token). */

/* Bits of ep_cfg_t.flags. */
#define EP_ZERO_PAD_ROWS 1u    /* also write zeros into the payload of pad rows */
/* ep_dispatch_layout path selection: at most one of the next four bits;
   every path gives the same results, they differ only in speed. */
#define EP_LAYOUT_LOOKBACK 2u  /* one kernel: ticketed tiles, each tile's prefix
                                  by decoupled look-back */
#define EP_LAYOUT_DIRECT 4u    /* two kernels: tile-count table, then ranks */
#define EP_LAYOUT_BARRIER 8u   /* one kernel: ticketed tiles, each tile's prefix
                                  from one read of every tile's counts; at
                                  most 2^20 routed slots (T*K), else
                                  EP_EINVAL: its cost grows with the square
                                  of the tile count */
#define EP_LAYOUT_COUNT 16u    /* one kernel: every workgroup counts every
                                  routed slot (no workspace traffic); at
                                  most 2^18 routed slots (T*K), else
                                  EP_EINVAL: its cost grows with the square
                                  of the batch */

/* Bits of the device flags word (ep_layout_t.flags[0]). */
#define EP_FLAG_DROPPED 1      /* a slot was dropped at segment capacity [TD]  */
#define EP_FLAG_BAD_ID 2       /* an expert id outside [-1, E) (slot masked)   */
#define EP_FLAG_INTERNAL 4     /* a layout row past recv_rows, or a single-pass
                                  wait gave up (neither happens in valid use) */
#define EP_FLAG_MAP_OVERFLOW 8 /* a routing-map row marked more than top_k experts */

/* Largest number of groups S * (E/S + shared_expert) a layout may have. */
#define EP_MAX_GROUPS 2048
/* Largest number of slots per token, K + shared_expert. */
#define EP_MAX_SLOTS 64

/*
 * Problem description.  Field names follow the pages' statement of the
 * problem ([MX] hidden_size, top_k, n_experts; [FA] num_local_experts,
 * pad_multiple, num_permuted_tokens).
 *
 * Groups: segment s has G = E/S + shared_expert groups.  With a fused
 * shared expert ([MX] fused_shared_expert) group 0 of every segment is the
 * shared group; only segment src_segment receives rows in it (every token
 * once, as top-k slot index `top_k`, expert id `num_experts`, weight 1 in
 * combine).  Routed expert e goes to segment e/(E/S), group shared+e%(E/S).
 */
typedef struct ep_cfg_t {
    int32_t num_tokens;    /* T >= 0 tokens of this GPU's share                   */
    int32_t hidden;        /* H >= 8, multiple of 8 (bf16 calls) or 16 (NVFP4)     */
    int32_t num_experts;   /* E >= 1 routed experts                               */
    int32_t num_segments;  /* S >= 1 destination segments, E % S == 0             */
    int32_t top_k;         /* K, 1 <= K <= E, K + shared_expert <= EP_MAX_SLOTS  */
    int32_t align;         /* A >= 1: each group's rows are padded to a multiple  */
    int32_t seg_capacity;  /* C >= 0: 0 = packed segments; > 0 = C rows per
                              segment, slots past it are dropped and flagged      */
    int32_t shared_expert; /* 0 or 1                                              */
    int32_t src_segment;   /* 0 <= src_segment < S (ignored without shared)       */
    int32_t reserved0;     /* must be 0                                           */
    int64_t recv_rows;     /* R: rows of every receive-side buffer (expert_ids,
                              src_info, recv, codes, ...); R >= ep_query's
                              min_recv_rows and R < 2^31.  A host integer, so no
                              call ever reads a count back from the device [FA]. */
    uint32_t flags;        /* EP_ZERO_PAD_ROWS, at most one EP_LAYOUT_* bit, or 0 */
    uint32_t reserved1;    /* must be 0                                           */
} ep_cfg_t;

/*
 * The dispatch "handle" ([FA] handle; [TD] overflow flag kept last): device
 * arrays written by ep_dispatch_layout and read by every later call.  K' =
 * K + shared_expert, G = groups per segment, R = recv_rows.
 *   counts         int32 [S*G]      valid slots per group ([TD] tokens per expert)
 *   seg_base       int32 [S+1]      first row of each segment (packed: running
 *                                   sum of used rows; capacity: s*C)
 *   row_offsets    int32 [S*(G+1)]  per segment, exclusive prefix of the
 *                                   aligned group sizes, clamped to C ([MX])
 *   scales_offsets int32 [S*(G+1)]  offsets into the block-scale rows; scales
 *                                   are row-major, so equal to row_offsets ([MX])
 *   token_row      int32 [T*K']     receive row of slot (t,k); -1 if the slot
 *                                   is masked, invalid or dropped ([TD] the
 *                                   reversed mapping used by combine)
 *   expert_ids     int32 [R]        expert of every used row, -1 on pad rows;
 *                                   shared rows carry E ([MX])
 *   src_info       int32 [R*2]      (token t, slot k) of every used row,
 *                                   (-1,-1) on pad rows ([MX])
 *   flags          int32 [1]        EP_FLAG_* bits for this dispatch ([TD])
 * Rows of a segment past its used rows are not written.  Within a group,
 * rows follow ascending slot index t*K'+k (stable, deterministic).
 */
typedef struct ep_layout_t {
    int32_t* counts;
    int32_t* seg_base;
    int32_t* row_offsets;
    int32_t* scales_offsets;
    int32_t* token_row;
    int32_t* expert_ids;
    int32_t* src_info;
    int32_t* flags;
} ep_layout_t;

/*
 * Sizes the caller must allocate for `cfg` (host only, no device work).
 *   min_recv_rows   packed: T*K' + min(T*K', E+shared)*(A-1) (every group
 *                   padded by at most A-1 rows, [TD] _align_up); capacity:
 *                   S*C.
 *   workspace_bytes scratch device memory for ep_dispatch_layout.
 *   groups_per_seg  G = E/S + shared_expert.
 * Any output pointer may be NULL.  Returns EP_OK or EP_EINVAL; recv_rows is
 * not checked here.
 */
int ep_query(const ep_cfg_t* cfg, int64_t* min_recv_rows, int64_t* workspace_bytes,
             int32_t* groups_per_seg);

/*
 * Build the receive layout from top-k expert ids ([FA] HybridEPDispatch
 * routing-metadata preprocessing; [TD] dispatch_postprocess counts;
 * [MX] row_offsets, expert_ids, src_info).
 *   topk_ids   int32 [T*K], row-major; -1 = unused slot ([FA] topk_idx)
 *   workspace  >= workspace_bytes from ep_query, 16-byte aligned, zero-filled
 *              before its first use; every call leaves it ready for the
 *              next one (reuse it: the single-pass kernels keep a generation
 *              count and a ticket in it).  Not shared by calls that may run
 *              at the same time.
 *   layout     the arrays above, all written here (src_info 8-byte aligned)
 * Steps: per tile of routed slots, a wavefront ballot/popcount histogram
 * and in-group ranks (stable, ascending slot index); each tile's prefix
 * over earlier tiles; the aligned group sizes scanned into group start rows;
 * token_row, expert_ids and src_info written.  Paths (same results):
 *  - up to 512 routed slots: one kernel in which every workgroup ranks
 *    all slots itself;
 *  - up to 8192 routed slots (by default; EP_LAYOUT_COUNT at any size): one
 *    kernel in which every workgroup counts all slots per group in LDS,
 *    then ranks its own tile;
 *  - otherwise (by default; EP_LAYOUT_DIRECT at any size): two kernels, a
 *    [tile][group] count table then the ranks, with a third launch between
 *    them past 256 tiles that sums the table in chunks of 256 tiles;
 *  - EP_LAYOUT_LOOKBACK / EP_LAYOUT_BARRIER: one kernel, tiles taken from
 *    an atomic ticket, each tile's prefix by decoupled look-back (or from
 *    one read of every tile's counts, whose cost grows with the square of
 *    the tile count); slower than the two kernels at every size measured.
 * At most 2^24 routed slots (T*K), else EP_EINVAL: up to there every path
 * costs about linearly in the slots (the single pass runs at most 8192
 * tiles).  The other calls take any T*K' < 2^30 with a valid token_row.
 * Data errors go to layout->flags; a single-pass wait that cannot end gives
 * up after about 0.3 s and sets EP_FLAG_INTERNAL.
 */
int ep_dispatch_layout(const ep_cfg_t* cfg, const int32_t* topk_ids, void* workspace,
                       int64_t workspace_bytes, const ep_layout_t* layout, void* stream);

/*
 * bf16 dispatch ([FA] HybridEPDispatch.forward with fuse_permute):
 *   recv[token_row[t,k], :] = x[t, :] bit for bit, for every kept slot.
 *   x     bf16 [T, H];  recv  bf16 [R, H].
 * Uses layout->token_row (and counts/row_offsets/seg_base when
 * EP_ZERO_PAD_ROWS is set).  Unused rows of recv are not written.
 */
int ep_dispatch(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* x,
                uint16_t* recv, void* stream);

/*
 * Layout and bf16 dispatch in one call ([FA] HybridEPDispatch.forward: the
 * permutation and the dispatch of one batch in a single call).  Same
 * arguments, outputs and errors as ep_dispatch_layout followed by
 * ep_dispatch on the same stream, and the same results bit for bit.  Up to
 * 512 routed slots (T*K; decode-sized batches) with no EP_LAYOUT_* path
 * flag, one kernel computes the layout and copies the payload rows: every
 * workgroup already ranks all slots there, so the copy needs no second
 * launch.  Larger batches, or a forced path, run the layout launches and
 * then the dispatch scatter.
 */
int ep_dispatch_with_layout(const ep_cfg_t* cfg, const int32_t* topk_ids, void* workspace,
                            int64_t workspace_bytes, const ep_layout_t* layout, const uint16_t* x,
                            uint16_t* recv, void* stream);

/*
 * NVFP4 dispatch with a per-token dynamic global scale ([MX] execute):
 * every token is quantized once and its bytes written to each kept row.
 *   x         bf16 [T, H] (H % 16 == 0)
 *   codes     uint8 [R, H/2]   E2M1 element codes, element 2j in the low
 *                              nibble of byte j, 2j+1 in the high nibble
 *   scales    uint8 [R, H/16]  E4M3 block scale of each 16-element block
 *   rowscale  bf16  [R]        bf16(1/g), the inverse global scale
 * Per token, in IEEE fp32 with round-to-nearest-even:
 *   rowmax = max|x|;  g = 2688 / rowmax;
 *   per block: s = (bmax / 6) * g -> E4M3 (RNE, saturating to 448);
 *              v = x * (g / e4m3(s)) -> E2M1 (RNE, ties to even, saturating
 *              at 6, sign bit of v kept); zero scale -> zero codes.
 *   An all-zero token gives zero codes, zero scales and rowscale +0.
 * Tokens must be finite; a token with 0 < rowmax < 2688/FLT_MAX (where g
 * overflows) is outside the contract.
 */
int ep_dispatch_nvfp4(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* x,
                      uint8_t* codes, uint8_t* scales, uint16_t* rowscale, void* stream);

/*
 * Layout and NVFP4 dispatch in one call ([MX] execute: the expert layout,
 * the per-token global scales and the NVFP4 payload of one batch in a
 * single call).  Same arguments, outputs and errors as ep_dispatch_layout
 * followed by ep_dispatch_nvfp4 on the same stream, and the same results
 * bit for bit.  Up to 512 routed slots (T*K) with no EP_LAYOUT_* path flag,
 * one kernel computes the layout and quantizes each token once into LDS,
 * then stores its codes, block scales and rowscale to each of its rows;
 * larger batches, or a forced path, run the layout launches and then the
 * NVFP4 dispatch.
 */
int ep_dispatch_nvfp4_with_layout(const ep_cfg_t* cfg, const int32_t* topk_ids, void* workspace,
                                  int64_t workspace_bytes, const ep_layout_t* layout, const uint16_t* x,
                                  uint8_t* codes, uint8_t* scales, uint16_t* rowscale, void* stream);

/*
 * FP8 dispatch ([FA] init_hybrid_ep_buffer: FP8 communication in the
 * dispatch phase; HybridEPDispatch.forward returns a scaling factor beside
 * the hidden states).  The pages give no format; this library reads it as
 * E4M3 codes with one fp32 factor per token and 128-element block:
 *   x       bf16 [T, H] (H % 128 == 0, H <= 16384)
 *   codes   uint8 [R, H]       E4M3 ("fn") codes
 *   scales  float [R, H/128]   dequantization factors
 * Per block, in IEEE fp32 with round-to-nearest-even: amax = max|x|;
 *   codes = E4M3(x * (448 / amax))  (saturating to 448, sign of the product kept)
 *   scale = amax / 448
 * An all-zero block gives zero codes and scale 0.  Every copy of a token
 * carries the same bytes.  Blocks with 0 < amax < 448/FLT_MAX are outside
 * the contract.
 */
int ep_dispatch_fp8(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* x,
                    uint8_t* codes, float* scales, void* stream);

/*
 * Layout and FP8 dispatch in one call ([FA] HybridEPDispatch.forward: the
 * permutation and the FP8 payload with its scaling factor from one call).
 * Same arguments, outputs and errors as ep_dispatch_layout followed by
 * ep_dispatch_fp8 on the same stream, and the same results bit for bit.  Up
 * to 512 routed slots (T*K) with no EP_LAYOUT_* path flag, one kernel
 * computes the layout and quantizes each token once per run of its rows,
 * storing codes and block scales to each; larger batches, or a forced path,
 * run the layout launches and then the FP8 dispatch.
 */
int ep_dispatch_fp8_with_layout(const ep_cfg_t* cfg, const int32_t* topk_ids, void* workspace,
                                int64_t workspace_bytes, const ep_layout_t* layout, const uint16_t* x,
                                uint8_t* codes, float* scales, void* stream);

/*
 * Combine ([FA] HybridEPCombine.forward; [TD] moe_router_dtype fp32):
 *   y[t, :] = bf16_rne( sum_{k=0..K'-1, token_row[t,k] >= 0}
 *                       w_k * float(expert_out[token_row[t,k], :]) )
 * accumulated in fp32 in ascending k, one rounding per multiply and per add
 * (no fused multiply-add), starting from +0.  w_k = probs[t,k] for routed
 * slots (1 when probs is NULL) and 1 for the shared slot.
 *   expert_out bf16 [R, H];  probs float [T, K] or NULL;  y bf16 [T, H].
 * Pad and dropped rows are never read.
 */
int ep_combine(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* expert_out,
               const float* probs, uint16_t* y, void* stream);

/*
 * Combine over NVFP4 expert-output rows ([MX] execute: the NVFP4 row format,
 * output_scales, output_rowwise_scales; [TD] moe_router_dtype fp32): the
 * expert outputs come back in the dispatch's NVFP4 format and are
 * dequantized as they are read:
 *   xhat = e2m1(code) * (e4m3(scale[h/16]) * float(rowscale[row]))
 *   y[t, h] = bf16_rne( sum_{k, token_row[t,k] >= 0} w_k * xhat(token_row[t,k], h) )
 * each product an fp32 multiply, accumulated in fp32 in ascending k from +0
 * with no fused multiply-add; w_k as in ep_combine.
 *   codes     uint8 [R, H/2]   element 2j in the low nibble of byte j (8-byte aligned)
 *   scales    uint8 [R, H/16]  E4M3 block scales, sign bit decoded; the NaN
 *                              codes 0x7F / 0xFF are outside the contract
 *   rowscale  bf16  [R]
 *   probs     float [T, K] or NULL;  y  bf16 [T, H]  (H % 16 == 0)
 * Pad and dropped rows are never read.  Returns EP_EINVAL past one grid:
 * T * ceil(H/1024) waves of 64 work-items must stay below 2^32.
 */
int ep_combine_nvfp4(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint8_t* codes, const uint8_t* scales,
                     const uint16_t* rowscale, const float* probs, uint16_t* y, void* stream);

/*
 * Dispatch backward ([FA] HybridEPDispatch.backward: combine the
 * gradients): grad_x[t] = bf16_rne( sum_k float(grad_recv[token_row[t,k]]) ),
 * fp32, ascending k, unweighted (dispatch is a copy); 0 if no slot is kept.
 *   grad_recv bf16 [R, H];  grad_x bf16 [T, H].
 */
int ep_dispatch_bwd(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* grad_recv,
                    uint16_t* grad_x, void* stream);

/*
 * Combine backward ([FA] HybridEPCombine.backward: redispatch through the
 * saved layout): grad_expert_out[token_row[t,k]] = bf16_rne(w_k * float(grad_y[t]))
 * for every kept slot, w_k as in ep_combine.
 *   grad_y bf16 [T, H];  probs float [T, K] or NULL;  grad_expert_out bf16 [R, H].
 */
int ep_combine_bwd(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* grad_y,
                   const float* probs, uint16_t* grad_expert_out, void* stream);

/*
 * Router-probability gradient ([FA] HybridEPDispatch.backward returns a
 * probability gradient beside the hidden-state gradient): with combine
 * y[t] = sum_k p[t,k] * out[row(t,k)],
 *   grad_probs[t,k] = <grad_y[t], expert_out[token_row[t,k]]>  (k < K)
 * as an fp32 dot product over H; 0 for masked, invalid and dropped slots.
 * The summation order is fixed (each of 256 threads sums its strided
 * share of the row in order, then a fixed tree), so results are
 * deterministic; they equal the exact dot product to within about
 * (8*ceil(H/2048) + 10) * 2^-24 * sum_h |grad_y[t,h] * out[row,h]|.
 *   grad_y bf16 [T, H];  expert_out bf16 [R, H];  grad_probs float [T, K].
 */
int ep_combine_bwd_probs(const ep_cfg_t* cfg, const ep_layout_t* layout, const uint16_t* grad_y,
                         const uint16_t* expert_out, float* grad_probs, void* stream);

/*
 * Compact top-k -> dense routing form ([TD] _HybridEPManager._indices_to_multihot;
 * [FA] HybridEPDispatch.forward accepts a Boolean routing map [tokens,
 * experts] with dense probabilities).  Only the fields T, E, K (and their
 * validity) of cfg are used.
 *   topk_ids     int32 [T, K]; -1 and ids outside [0, E) mark nothing
 *   probs        float [T, K]; required iff dense_probs is not NULL
 *   routing_map  uint8 [T, E]: 1 where some slot names the expert, else 0
 *   dense_probs  float [T, E] or NULL: sum of the probabilities of the slots
 *                naming the expert, added in slot order; 0 elsewhere
 */
int ep_indices_to_multihot(const ep_cfg_t* cfg, const int32_t* topk_ids, const float* probs,
                           uint8_t* routing_map, float* dense_probs, void* stream);

/*
 * Dense routing form -> compact top-k (the reverse; [FA] routing_map takes
 * precedence over topk_idx, so a caller holding both converts the map).
 *   routing_map  uint8 [T, E]; any nonzero byte marks the expert
 *   dense_probs  float [T, E]; required iff probs is not NULL
 *   topk_ids     int32 [T, K]: the marked experts in ascending order, then -1
 *   probs        float [T, K] or NULL: their dense probabilities, then 0
 *   flags        int32 [1] or NULL: OR-ed with EP_FLAG_MAP_OVERFLOW when a
 *                row marks more than K experts (the lowest K are kept); the
 *                caller clears it
 */
int ep_multihot_to_indices(const ep_cfg_t* cfg, const uint8_t* routing_map, const float* dense_probs,
                           int32_t* topk_ids, float* probs, int32_t* flags, void* stream);

/*
 * ep_dispatch_layout without a caller workspace, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same arguments, results and errors as
 * ep_dispatch_layout, except that the workspace is a buffer built into the
 * library: EP_NOALLOC_SCRATCH_BYTES bytes per GPU, held from the first call
 * on that GPU until the process ends.  Returns EP_ESCRATCH, before anything
 * is enqueued, when ep_query's workspace_bytes for cfg exceeds it.  Every
 * call on one GPU shares that buffer: two calls that may run at the same
 * time on one GPU (different streams, no ordering between them) race and
 * give undefined layouts; calls on one stream are ordered and safe.  Never
 * allocates, frees or synchronizes.
 */
#define EP_NOALLOC_SCRATCH_BYTES (4 << 20)
int ep_dispatch_layout_noalloc(const ep_cfg_t* cfg, const int32_t* topk_ids, const ep_layout_t* layout,
                               void* stream);

/* ------------------------------------------------------------------------
 * The expert layer: what runs between the router's logits and ep_combine.
 *   logits --ep_route--> topk_ids, probs --ep_dispatch_layout / ep_dispatch-->
 *   recv --ep_expert_gemm--> h --ep_swiglu (weights applied)--> act
 *   --ep_expert_gemm--> out --ep_combine (probs NULL)--> y
 * (or ep_swiglu with probs NULL and ep_combine with probs).  Rows that no
 * kept slot owns (pad rows, rows past a segment's used rows, rows of dropped
 * slots) are never read and, unless EP_ZERO_PAD_ROWS is set, never written.
 * No output of these calls may overlap an input (EP_GRAD_F32_ADD's grad_w is
 * both).
 * ------------------------------------------------------------------------ */

/* ep_route_t.score */
#define EP_SCORE_SOFTMAX 0  /* s = softmax of the token's logits over all experts */
#define EP_SCORE_SIGMOID 1  /* s = 1 / (1 + exp(-logit)), each expert by itself   */
/* ep_route_t.logits_type */
#define EP_TYPE_F32 0
#define EP_TYPE_BF16 1
/* Largest num_groups of ep_route_t. */
#define EP_MAX_ROUTE_GROUPS 64

/* How ep_route chooses and weights a token's experts. */
typedef struct ep_route_t {
    int32_t score;        /* EP_SCORE_*                                             */
    int32_t normalize;    /* 1: the chosen scores are divided by their sum + 1e-20  */
    int32_t num_groups;   /* >= 1, divides num_experts: experts [g*E/num_groups,
                             (g+1)*E/num_groups) form group g; <= EP_MAX_ROUTE_GROUPS */
    int32_t top_groups;   /* 1 <= top_groups <= num_groups: experts are chosen from
                             this many groups                                       */
    float scale;          /* finite; multiplies every weight                        */
    int32_t logits_type;  /* EP_TYPE_*: type of logits (and of their gradient)      */
    int32_t reserved0;    /* must be 0                                              */
    int32_t reserved1;    /* must be 0                                              */
} ep_route_t;

/*
 * Router: the experts and weights of every token ([TD] moe_router_dtype: fp32
 * routing weights; [FA] topk_idx with -1 for unused slots, topk_weights).
 *   logits      [T, E] of route->logits_type
 *   bias        float [E] or NULL: added to the scores for the choice only
 *   token_mask  uint8 [T] or NULL: tokens with 0 get no experts
 *   topk_ids    int32 [T, K]   the chosen experts, best first; what
 *                              ep_dispatch_layout takes
 *   probs       float [T, K]   their weights; what ep_combine / ep_swiglu take
 * key = s + bias where there is a bias, the logit itself where there is none
 * (the scores grow with it).  A group's key is the sum of its two largest
 * keys with a bias (its only key in a group of one) and its largest key
 * without; the top_groups groups with the largest keys stay.  The K experts
 * of the largest keys among them are chosen; ties go to the lower index, of
 * groups and of experts.  Keys with a bias are ordered as 64-bit floating
 * point orders them: two experts are told apart where fp32 scores would round
 * to the same value.
 *   probs[t,k] = scale * s[id_k] / (sum_j s[id_j] + 1e-20)   normalize = 1
 *              = scale * s[id_k]                             normalize = 0
 * in fp32, from the scores without the bias.
 * logits and grad_logits are 16-byte aligned.
 * An expert with a logit of -infinity or NaN is never chosen; a token with
 * fewer than K experts to choose from has id -1 and weight 0 in its last
 * slots.  Softmax sums over every expert of the token: a NaN or +infinity
 * among its logits makes its weights NaN, and its experts are chosen as without
 * a bias.  bias is finite.
 * Only T, E, K (and their validity) of cfg are used.
 */
int ep_route(const ep_cfg_t* cfg, const ep_route_t* route, const void* logits, const float* bias,
             const uint8_t* token_mask, int32_t* topk_ids, float* probs, void* stream);

/*
 * Router backward: the gradient of ep_route's weights with respect to the
 * logits, the choice held fixed (the bias gets none).
 *   logits      [T, E] of route->logits_type, as in the forward call
 *   topk_ids    int32 [T, K]   ep_route's; -1 and ids outside [0, E) count as
 *                              unused slots (grad_probs is not read into them)
 *   grad_probs  float [T, K]
 *   grad_logits [T, E] of route->logits_type, all written; 0 for a token
 *               without experts
 * With q_k = s[id_k], Q = sum q + 1e-20 and the weights' gradient g:
 *   gq_k = scale * (g_k - sum_j g_j q_j / Q) / Q (normalize), scale * g_k (not)
 *   sigmoid: grad_logits[id_k] = gq_k q_k (1 - q_k), 0 elsewhere
 *   softmax: grad_logits[e] = s_e (sum_{k: id_k = e} gq_k - sum_j gq_j q_j)
 * in fp32, rounded once to the logits' type.
 */
int ep_route_bwd(const ep_cfg_t* cfg, const ep_route_t* route, const void* logits, const int32_t* topk_ids,
                 const float* grad_probs, void* grad_logits, void* stream);

/*
 * Gated activation on the receive rows, with the routing weights applied to
 * the sorted rows ([FA] HybridEPDispatch.forward hands the experts their rows'
 * probabilities): for every kept slot, row r = token_row[t,k],
 *   act[r, i] = bf16_rne( w * (silu(h[r, i]) * h[r, inter + i]) )
 * silu(a) = a / (1 + exp(-a)), in fp32; w = probs[t,k] for routed slots (1
 * when probs is NULL) and 1 for the shared slot.
 *   h    bf16 [R, 2*inter]  (gate, then up; inter >= 8, a multiple of 8)
 *   probs float [T, K] or NULL;  act  bf16 [R, inter]
 */
int ep_swiglu(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t inter, const uint16_t* h,
              const float* probs, uint16_t* act, void* stream);

/*
 * Backward of ep_swiglu: for every kept slot, with a, b the row's two halves,
 * s = 1 / (1 + exp(-a)) and g the row of grad_act, in fp32,
 *   grad_h[r, i]         = bf16_rne( w g b s (1 + a (1 - s)) )
 *   grad_h[r, inter + i] = bf16_rne( w g a s )
 *   grad_probs[t, k]     = sum_i g a s b      (k < K; 0 for masked, invalid and
 *                          dropped slots), summed in a fixed order
 *   grad_probs float [T, K], or NULL to leave it out.
 * grad_h may not overlap h or grad_act.
 */
int ep_swiglu_bwd(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t inter, const uint16_t* h,
                  const float* probs, const uint16_t* grad_act, uint16_t* grad_h, float* grad_probs,
                  void* stream);

/* Largest in_dim and out_dim of the experts' products. */
#define EP_MAX_EXPERT_DIM (1 << 20)

/*
 * The experts' product: every kept row times its own expert's weights,
 *   y[r, n] = bf16_rne( sum_h x[r, h] w[e(r), n, h] )   (fp32 accumulation)
 *   x  bf16 [R, in_dim];  w  bf16 [E + shared_expert, out_dim, in_dim], the
 *   shared expert last;  y  bf16 [R, out_dim].
 * in_dim and out_dim: multiples of 8 in [8, EP_MAX_EXPERT_DIM] (cfg->hidden
 * takes no part).  Uses layout->counts, row_offsets and seg_base, not the
 * ids: rows of one group belong to one expert.  A row's results do not depend
 * on which other rows its group holds, and repeat bit for bit.  This call, its
 * gradients and ep_expert_gemm_nvfp4 return EP_EINVAL where their tiles pass
 * one grid of 2^32 work-items (2^23 tiles of 128 x 256 results; 2^24 tiles of
 * 16 x 64 for 4-bit weights).
 */
int ep_expert_gemm(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t in_dim, int32_t out_dim,
                   const uint16_t* x, const uint16_t* w, uint16_t* y, void* stream);

/*
 * The input's gradient of ep_expert_gemm:
 *   grad_x[r, h] = bf16_rne( sum_n grad_y[r, n] w[e(r), n, h] )
 */
int ep_expert_gemm_bwd_x(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t in_dim, int32_t out_dim,
                         const uint16_t* grad_y, const uint16_t* w, uint16_t* grad_x, void* stream);

/* How ep_expert_gemm_bwd_w leaves the weights' gradient. */
#define EP_GRAD_BF16 0     /* grad_w bf16, overwritten                           */
#define EP_GRAD_F32 1      /* grad_w float, overwritten                          */
#define EP_GRAD_F32_ADD 2  /* grad_w float, added to (gradients over several batches) */

/*
 * The weights' gradient of ep_expert_gemm:
 *   grad_w[e, n, h] = sum_{r of expert e} grad_y[r, n] x[r, h]   (fp32 accumulation)
 * for all E + shared_expert experts; one without rows gets zeros (EP_GRAD_F32_ADD:
 * stays as it is).  The order of the sum is fixed: results repeat bit for bit.
 */
int ep_expert_gemm_bwd_w(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t in_dim, int32_t out_dim,
                         const uint16_t* grad_y, const uint16_t* x, void* grad_w, int32_t grad_type, void* stream);

/*
 * The experts' product over 4-bit weights, in the dispatch's NVFP4 row format
 * ([MX]): w[e, n, h] = e2m1(code) * e4m3(scales[e, n, h/16]) * float(rowscale[e, n]),
 *   y[r, n] = bf16_rne( float(rowscale[e, n]) * sum_h x[r, h] * e2m1 * e4m3 )
 * (the product of a code and its block scale is exact; fp32 accumulation).
 *   x        bf16  [R, in_dim]
 *   codes    uint8 [E + shared, out_dim, in_dim/2]   element 2j in the low nibble
 *   scales   uint8 [E + shared, out_dim, in_dim/16]  E4M3, sign bit decoded; the NaN
 *                                                    codes 0x7F / 0xFF are outside the contract
 *   rowscale bf16  [E + shared, out_dim]
 *   y        bf16  [R, out_dim]
 * in_dim: a multiple of 16, out_dim of 8, both at most EP_MAX_EXPERT_DIM; codes
 * and scales 16-byte aligned, rowscale 8-byte.
 */
int ep_expert_gemm_nvfp4(const ep_cfg_t* cfg, const ep_layout_t* layout, int32_t in_dim, int32_t out_dim,
                         const uint16_t* x, const uint8_t* codes, const uint8_t* scales,
                         const uint16_t* rowscale, uint16_t* y, void* stream);

/* ------------------------------------------------------------------------
 * Low-rank adapters of many requests beside the experts' products: a row of
 * expert e and of a token with adapter d has
 *   u = scale[d] A[d, e] x,   y = w[e] x + B[d, e] u
 * and a row of a token without one y = w[e] x.  ep_lora_down makes u; the
 * products below take it and B.  Every adapter reaches its own rows alone,
 * infinities and NaN in it included.
 * ------------------------------------------------------------------------ */
#define EP_MAX_LORA_RANK 128
#define EP_MAX_ADAPTERS 65536

typedef struct ep_lora_t {
    const int32_t* token_adapter; /* int32 [T]: the adapter of each token; -1 and ids
                                     outside [0, num_adapters): none                 */
    const uint16_t* a;            /* bf16 [num_adapters, E + shared_expert, rank, in_dim]  */
    const uint16_t* b;            /* bf16 [num_adapters, E + shared_expert, out_dim, rank] */
    const float* scale;           /* float [num_adapters], or NULL: 1                */
    int32_t num_adapters;         /* 1 .. EP_MAX_ADAPTERS                            */
    int32_t rank;                 /* a multiple of 8 in [8, EP_MAX_LORA_RANK]        */
    int32_t reserved0;            /* must be 0                                       */
    int32_t reserved1;            /* must be 0                                       */
} ep_lora_t;
/* a, b and u are 16-byte aligned.  in_dim, out_dim and w are the product's they
 * stand beside; a call checks and reads a, b and scale only as its formula names
 * them.  All of these calls read counts, row_offsets, seg_base and src_info of the
 * layout, with token_adapter as it was for ep_lora_down. */

/*
 * u[r] = scale[d] A[d, e(r)] x[r] for every kept row (fp32 accumulation), zeros
 * for those without an adapter.
 *   x  bf16 [R, in_dim]
 *   u  float [R, rank]; the products take it as two bf16 a value (16 significant
 *      bits), the adapters' gradients as three (24).  An infinity times u is one of
 *      that sign all the same (NaN where u is 0, or below half of bf16's smallest).
 */
int ep_lora_down(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                 const uint16_t* x, float* u, void* stream);

/* ep_expert_gemm with the adapters' part:
 *   y[r, n] = bf16_rne( sum_h x[r, h] w[e(r), n, h] + sum_p B[d, e(r), n, p] u[r, p] ) */
int ep_expert_gemm_lora(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                        int32_t out_dim, const uint16_t* x, const uint16_t* w, const float* u, uint16_t* y, void* stream);

/* ep_expert_gemm_nvfp4 with the adapters' part (in bf16 beside the 4-bit weights). */
int ep_expert_gemm_nvfp4_lora(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                              int32_t out_dim, const uint16_t* x, const uint8_t* codes, const uint8_t* scales,
                              const uint16_t* rowscale, const float* u, uint16_t* y, void* stream);

/* grad_u[r] = scale[d] B[d, e(r)]^T grad_y[r], held as u is; zeros for rows
 * without an adapter. */
int ep_lora_bwd_u(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t out_dim,
                  const uint16_t* grad_y, float* grad_u, void* stream);

/* ep_expert_gemm_bwd_x with the adapters' part:
 *   grad_x[r, h] = bf16_rne( sum_n grad_y[r, n] w[e(r), n, h] + sum_p A[d, e(r), p, h] grad_u[r, p] ) */
int ep_expert_gemm_bwd_x_lora(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                              int32_t out_dim, const uint16_t* grad_y, const uint16_t* w, const float* grad_u,
                              uint16_t* grad_x, void* stream);

/*
 * The adapters' gradients, over the rows r of expert e whose tokens have adapter d:
 *   grad_a[d, e, p, h] = sum_r grad_u[r, p] x[r, h]     [num_adapters, E + shared, rank, in_dim]
 *   grad_b[d, e, n, p] = sum_r grad_y[r, n] u[r, p]     [num_adapters, E + shared, out_dim, rank]
 * both of grad_type (EP_GRAD_*: bf16, float, float added to), zeros where no row
 * is.  Sums in row order: results repeat bit for bit.  (scale is part of u and
 * grad_u; a and b of lora are not read.)  Returns EP_EINVAL past one grid of 2^32
 * work-items, 2^24 tiles of 256 columns of either over all adapters and experts; neither
 * is written then.
 */
int ep_lora_bwd_w(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                  int32_t out_dim, const uint16_t* x, const uint16_t* grad_y, const float* u, const float* grad_u,
                  void* grad_a, void* grad_b, int32_t grad_type, void* stream);

/*
 * The gated block in one kernel: both projections, the activation and the
 * routing weight (ep_expert_gemm over the stacked weights and ep_swiglu, without
 * h in between: g and u below are not rounded).
 *   g = sum_h x[r, h] w[e(r), i, h],  u = sum_h x[r, h] w[e(r), inter + i, h]
 *   act[r, i] = bf16_rne( w_r * (silu(g) * u) )
 *   x     bf16 [R, in_dim];  w  bf16 [E + shared_expert, 2*inter, in_dim] (gate rows, then up rows)
 *   probs float [T, K] or NULL (w_r = 1; 1 in the shared slot as well);  act  bf16 [R, inter]
 *   lora  NULL, or adapters beside the stacked weights (B [.., 2*inter, rank]), added to g
 *         and u before the activation; ulora: ep_lora_down's of x (NULL without)
 * in_dim and inter: multiples of 8 in [8, EP_MAX_EXPERT_DIM] (2*inter at most that where
 * gradients of x and w are to follow).  Reads counts,
 * row_offsets, seg_base and src_info of the layout.
 */
int ep_expert_gated(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim, int32_t inter,
                    const uint16_t* x, const uint16_t* w, const float* probs, const float* ulora, uint16_t* act,
                    void* stream);

/* The same over 4-bit weights, as in ep_expert_gemm_nvfp4 with out_dim 2*inter
 * (in_dim a multiple of 16, inter * in_dim < 2^34). */
int ep_expert_gated_nvfp4(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                          int32_t inter, const uint16_t* x, const uint8_t* codes, const uint8_t* scales,
                          const uint16_t* rowscale, const float* probs, const float* ulora, uint16_t* act, void* stream);

/* Columns of act whose share of grad_probs is one part of the workspace. */
#define EP_GATED_PART 32

/*
 * Backward of ep_expert_gated, which makes g and u again (neither is kept
 * between the passes): with s = 1 / (1 + exp(-g)) and ga the row of grad_act, in fp32,
 *   grad_h[r, i]         = bf16_rne( w_r ga u s (1 + g (1 - s)) )
 *   grad_h[r, inter + i] = bf16_rne( w_r ga g s )
 *   grad_probs[t, k]     = sum_i ga silu(g) u   (k < K; 0 for masked, invalid and dropped
 *                          slots; float [T, K], or NULL to leave it out)
 *   act                  as the forward pass, or NULL to leave it out
 * and, from grad_h, the gradients of x and w by ep_expert_gemm_bwd_x and
 * ep_expert_gemm_bwd_w (of the adapters by ep_lora_bwd_u and ep_lora_bwd_w).  A training
 * step of ep_expert_gemm and ep_swiglu with their backward calls keeps h and takes less time.
 *   grad_act bf16 [R, inter];  grad_h bf16 [R, 2*inter]
 *   workspace: with grad_probs, at least T * K * ceil(inter / EP_GATED_PART) * 4
 *              bytes, 16-byte aligned, of any content; not shared by calls that may
 *              run at the same time.  Else NULL.
 */
int ep_expert_gated_bwd(const ep_cfg_t* cfg, const ep_layout_t* layout, const ep_lora_t* lora, int32_t in_dim,
                        int32_t inter, const uint16_t* x, const uint16_t* w, const float* probs, const float* ulora,
                        const uint16_t* grad_act, uint16_t* grad_h, uint16_t* act, float* grad_probs, void* workspace,
                        int64_t workspace_bytes, void* stream);

/* Static description of a status code. */
const char* ep_strerror(int status);

/* EPX_ABI_VERSION of the built library. */
int ep_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* EPX_H */
