/*
 * moe.h -- C ABI of the GB300 (sm_103a) MoE layer forward.
 *
 * The layer computes y = sum_{i in TopK(x)} g_i(x) * E_i(x) (+ an optional
 * shared expert), each E_i a SwiGLU FFN ("TensorRT-LLM 源码完全拆解(十三): MoE 层前向执行",
 * section "MoE 在推理侧到底特殊在哪里"), in five steps:
 *
 *   1. moe_route     router logits -> (token_selected_experts, token_final_scales)
 *   2. moe_permute   rows of x gathered into contiguous per-expert blocks
 *   3. moe_fc1       grouped GEMM x_perm . w13[e]^T with SwiGLU fused -> h
 *   4. moe_fc2       grouped GEMM h . w2[e]^T -> out_perm
 *      (moe_fc1_fc2  steps 3 and 4 in one persistent launch, as moe_forward runs them)
 *   5. moe_finalize  unpermute, apply the routing weights, add the shared expert -> y
 *
 * moe_forward runs steps 2-5. Conventions common to every call:
 *
 *  - Pointers named "device" are CUDA device memory owned by the caller. The
 *    library allocates no device memory; the forward uses the caller's
 *    workspace (size from moe_workspace_bytes).
 *  - `stream` is a cudaStream_t (passed as void*). Work is enqueued on it
 *    only; no call below synchronises except moe_read_device_status and
 *    moe_static_read_device_status.
 *  - bf16 tensors are passed as void* to 2-byte IEEE bfloat16 elements,
 *    row-major, innermost dimension contiguous. Every device pointer must be
 *    16-byte aligned.
 *  - Errors found on the host (bad sizes, NULL or misaligned pointers, a
 *    workspace that is too small) return synchronously and enqueue nothing.
 *    A CUDA launch error returns MOE_ERR_CUDA (text in moe_last_error()).
 *    Errors found on the device (an expert id outside [0, E), a bounded wait
 *    that ran out) set bits in the workspace status word; the offending rows
 *    are skipped. moe_read_device_status reports them.
 *  - T = 0 is a valid no-op.
 *
 * Thread safety: calls may come from several host threads; calls that share
 * a workspace must be ordered on one stream.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ABI_VERSION 1

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,        /* NULL/misaligned pointer, negative size          */
  MOE_ERR_UNSUPPORTED = 2,        /* shape outside the supported envelope (reason)    */
  MOE_ERR_WORKSPACE_TOO_SMALL = 3,
  MOE_ERR_CUDA = 4,               /* a CUDA runtime call failed                       */
  MOE_ERR_DEVICE_BAD_ID = 5,      /* device saw an expert id outside [0, E)           */
  MOE_ERR_DEVICE_TIMEOUT = 6,     /* a bounded device-side wait ran out               */
  MOE_ERR_NOT_IMPLEMENTED = 7
} moe_status;

/* Routing methods; the values are those of the RoutingMethodType enum on the
 * TensorRT-LLM MoE page (section "路由方法枚举"). */
typedef enum {
  MOE_ROUTE_DEFAULT = 0,           /* softmax over E -> top-k, weights = selected probabilities   */
  MOE_ROUTE_RENORMALIZE = 1,       /* top-k -> softmax over the k selected logits                 */
  MOE_ROUTE_DEEPSEEKV3 = 2,        /* sigmoid, +bias for selection, top-2 per group, top groups,
                                      top-k; weights = unbiased sigmoid / (sum + 1e-20) * rsf    */
  MOE_ROUTE_LLAMA4 = 3,            /* top-k by logit ("Top1"), weights = sigmoid of each selected
                                      logit, not renormalised                                     */
  MOE_ROUTE_RENORMALIZE_NAIVE = 4, /* softmax over E -> top-k -> divide by the selected sum       */
  MOE_ROUTE_MINIMAX2 = 5,          /* sigmoid, +bias for selection, top-k over all E; weights =
                                      unbiased sigmoid / their sum (bias optional, NULL = 0)     */
  MOE_ROUTE_SIGMOID_RENORM = 6,    /* sigmoid -> top-k -> divide by the selected sum              */
  /* vLLM's GroupedTopKRouter (vLLM MoE page, section "GroupedTopKRouter：分组的专家选择"); the
   * values lie outside RoutingMethodType's range (0-8). */
  MOE_ROUTE_GROUPED_TOPK = 16,     /* sigmoid scores; group score = sum of the group's scores;
                                      top topk_group groups; top_k / topk_group experts inside
                                      each; weights = scores / their sum * rsf (see moe_route) */
  MOE_ROUTE_GROUPED_TOPK_SOFTMAX = 17  /* the same with a softmax inside each group: its group
                                      scores are all 1, so the group choice would rest on
                                      tie-breaking alone; always rejected (MOE_REASON_DEGENERATE) */
} moe_route_method;

/* Why moe_can_implement rejected a problem. */
typedef enum {
  MOE_REASON_OK = 0,
  MOE_REASON_T_RANGE = 1,          /* T < 0 or T > 2^24                                   */
  MOE_REASON_E_RANGE = 2,          /* E < 1 or E > 256                                    */
  MOE_REASON_TOPK_RANGE = 3,       /* k < 1 or k > 8                                      */
  MOE_REASON_H_ALIGN = 4,          /* H < 64, H % 64 != 0 or H > 32768                    */
  MOE_REASON_I_ALIGN = 5,          /* I < 64, I % 64 != 0 or I > 65536                    */
  MOE_REASON_SHARED_I_ALIGN = 6,   /* shared_I < 0, shared_I % 64 != 0 or > 65536         */
  MOE_REASON_GROUPS = 7,           /* routing groups invalid (see moe_route)              */
  MOE_REASON_METHOD = 8,           /* unknown routing method                              */
  MOE_REASON_ROWS = 9,             /* T*k (+T shared) permuted rows reach 2^31             */
  MOE_REASON_DEGENERATE = 10       /* a routing whose choice rests on tie-breaking alone   */
} moe_reason;

typedef struct {
  int32_t num_experts;            /* E                                                   */
  int32_t top_k;                  /* k                                                   */
  int32_t method;                 /* moe_route_method                                    */
  int32_t n_group;                /* DeepSeekV3, GROUPED_TOPK: expert groups; else 1      */
  int32_t topk_group;             /* DeepSeekV3, GROUPED_TOPK: groups kept; else 1        */
  float routed_scaling_factor;    /* DeepSeekV3, GROUPED_TOPK: multiplies the weights     */
} moe_route_params;

typedef struct {
  int64_t T;                      /* tokens                                              */
  int32_t H;                      /* hidden size                                         */
  int32_t I;                      /* routed expert intermediate size                     */
  int32_t E;                      /* routed experts                                      */
  int32_t k;                      /* experts per token                                   */
  int32_t shared_I;               /* shared expert intermediate size; 0 = no shared      */
} moe_problem;

/* Byte offsets of the workspace regions (all 1024-byte aligned). */
typedef struct {
  size_t status;      /* int32[4]: device status bits (MOE_DEVICE_FLAG_*)                    */
  size_t counts;      /* int32[G]: rows per group; G = E (+1 with a shared expert)           */
  size_t starts;      /* int32[G]: first permuted row of each group (shared group: T*k)      */
  size_t offsets;     /* int32[E+1]: exclusive scan of the routed counts                     */
  size_t tile_off1;   /* int32[2][G+1]: FC1 offsets per group, CTA-pair list then single-SM  */
  size_t tile_off2;   /* int32[2][G+1]: FC2 offsets per group, CTA-pair list then single-SM  */
  size_t sched;       /* int32[8 + G]: GEMM work-claim/finish counters, then per-group FC1 done  */
  size_t block_hist;  /* int32[nb*E]: per-chunk expert histograms                            */
  size_t perm_src;    /* int32[T*k]: permuted row -> flat index f = t*k + j                  */
  size_t perm_inv;    /* int32[T*k]: flat index -> permuted row (-1 if the id was invalid)   */
  size_t x_perm;      /* bf16[R, H]: gathered rows, R = T*k (+T shared rows)                 */
  size_t h;           /* bf16[R, Ih]: SwiGLU output, Ih = max(I, shared_I)                   */
  size_t out_perm;    /* bf16[R, H]: FC2 output in permuted order                            */
  size_t total;       /* bytes = moe_workspace_bytes()                                       */
  int64_t rows;       /* R                                                                   */
  int32_t groups;     /* G                                                                   */
  int32_t n_chunks;   /* nb                                                                  */
  int32_t h_ld;       /* Ih                                                                  */
  int32_t reserved;
} moe_ws_layout;

#define MOE_DEVICE_FLAG_BAD_ID 1
#define MOE_DEVICE_FLAG_TIMEOUT 2

int32_t moe_abi_version(void);
const char* moe_status_string(moe_status s);
/* Text of the last error seen on the calling host thread ("" if none). */
const char* moe_last_error(void);

/*
 * moe_route -- routing (step 1).
 * Source: TensorRT-LLM MoE page, sections "路由方法枚举" and "DeepSeek-V3 的 noaux_tc:
 * 分组路由的算术" (apply() returns token_selected_experts int32 [T, k] and
 * token_final_scales fp32 [T, k]); vLLM MoE page, section "FusedTopKRouter".
 *   logits  device fp32 [T, E] row-major.
 *   bias    device fp32 [E] e_score_correction_bias (DeepSeekV3), or NULL (= zeros).
 *   ids     device int32 [T, k] out: selected experts, by descending selection key,
 *           ties to the lower expert index. The key is the fp32 logit for the softmax
 *           and sigmoid methods; for DeepSeekV3 it is fl32(fl32(sigmoid_fp64(l)) + b).
 *   scales  device fp32 [T, k] out: routing weights (computed in fp64, rounded once).
 * Envelope (the fused-routing limits of the TensorRT-LLM page, section "融合算子与回退
 * 阈值"): 1 <= k <= 8, k <= E <= 256; DeepSeekV3 also E % n_group == 0, n_group <= 32,
 * 2 <= E/n_group <= 32, 1 <= topk_group <= n_group, k <= topk_group*E/n_group <= 256.
 * Outside it: MOE_ERR_UNSUPPORTED, nothing enqueued (there is no fallback).
 * Non-finite logits count as -inf for selection and in the normalisers.
 * MOE_ROUTE_GROUPED_TOPK (vLLM MoE page, section "GroupedTopKRouter"): score
 * s = sigmoid_fp64(l), key fl32(s); a group's score is the sum of its keys added in fp32
 * in expert order; the topk_group best groups (ties to the lower group index), then the
 * k / topk_group best keys inside each (ties to the lower index); slots by descending key;
 * weights s / sum(s) * routed_scaling_factor. Needs E % n_group == 0, n_group <= 32,
 * 1 <= topk_group <= n_group, k % topk_group == 0, k / topk_group <= E / n_group; `bias`
 * must be NULL (MOE_ERR_INVALID_ARG otherwise).
 */
moe_status moe_route(const float* logits, int64_t T, const float* bias, const moe_route_params* p,
                     int32_t* ids, float* scales, void* stream);

/* Pure check of a problem against the supported envelope; never touches the device.
 * Returns MOE_OK or MOE_ERR_UNSUPPORTED / MOE_ERR_INVALID_ARG; *reason (may be NULL)
 * receives a moe_reason. */
moe_status moe_can_implement(const moe_problem* p, int32_t* reason);

/* Workspace bytes the forward needs for this problem (0 if it is unsupported). */
size_t moe_workspace_bytes(const moe_problem* p);
/* Fills *out with the workspace layout for this problem. */
moe_status moe_workspace_layout(const moe_problem* p, moe_ws_layout* out);

/*
 * moe_forward -- steps 2-5 on one stream.
 * Source: vLLM MoE page, section "Router 的子类选择逻辑"/"量化与 MoE Kernel 选择" (the
 * modular path forward_modular(x, topk_weights, topk_ids)) and section "专家权重如何存储"
 * (w13 = gate and up merged [E, 2I, H], w2 = down [E, H, I]); TensorRT-LLM MoE page,
 * layer-structure figure (routed path + shared expert summed).
 *   x        device bf16 [T, H]
 *   ids      device int32 [T, k] (any values; ids outside [0, E) are skipped and flagged;
 *            repeated ids in a row are independent rows)
 *   scales   device fp32 [T, k]
 *   w13      device bf16 [E, 2I, H]: rows [0, I) gate (w1), rows [I, 2I) up (w3)
 *   w2       device bf16 [E, H, I]
 *   w13_s    device bf16 [2*shared_I, H] or NULL when shared_I == 0
 *   w2_s     device bf16 [H, shared_I]  or NULL when shared_I == 0
 *   y        device bf16 [T, H] out: sum_j scales[t,j] * E_ids[t,j](x[t]) + shared(x[t])
 *   workspace device, >= moe_workspace_bytes(p) bytes, 1024-byte aligned.
 * Accumulation is fp32; h and out_perm are rounded to bf16; y is rounded once to bf16.
 */
moe_status moe_forward(const moe_problem* p, const void* x, const int32_t* ids, const float* scales,
                       const void* w13, const void* w2, const void* w13_s, const void* w2_s,
                       void* y, void* workspace, size_t ws_bytes, void* stream);

/*
 * moe_forward_static -- moe_forward without a caller workspace. The pages have no
 * counterpart; this entry point exists for callers that cannot allocate device memory:
 * plugins hosted by an inference engine that owns every device allocation, and
 * latency-critical loops that must not call cudaMalloc (it can synchronise the whole
 * device). The scratch the forward needs lives in a fixed array inside this library,
 * MOE_STATIC_SCRATCH_BYTES bytes on every GPU that loads it, held until the process
 * exits. Arguments are those of moe_forward minus the workspace.
 *  - Problems whose workspace (moe_workspace_bytes) exceeds MOE_STATIC_SCRATCH_BYTES are
 *    rejected with MOE_ERR_WORKSPACE_TOO_SMALL before anything is enqueued.
 *  - The first call on a device looks up the array's device address (once per device,
 *    with that device current); make that first call before any stream capture.
 *  - Every call on a device shares the one array and it keeps the previous call's
 *    contents (the call clears what must start at zero itself). Calls whose work
 *    overlaps on the GPU race: order them on one stream.
 *  - Device-detected errors (ids outside [0, E), a bounded wait that ran out) skip rows
 *    as in moe_forward and set the status word inside the array, which each call clears
 *    when it starts; moe_static_read_device_status reads it back.
 * It allocates nothing: no cudaMalloc, no cudaFree, no allocating library routine.
 */
#define MOE_STATIC_SCRATCH_BYTES ((size_t)32 << 20)
moe_status moe_forward_static(const moe_problem* p, const void* x, const int32_t* ids,
                              const float* scales, const void* w13, const void* w2,
                              const void* w13_s, const void* w2_s, void* y, void* stream);

/* The status word of moe_forward_static on the current device: synchronises `stream`
 * (the stream the forward ran on), reads and clears the word inside the library's
 * scratch array. *flags (may be NULL) receives the MOE_DEVICE_FLAG_* bits. Returns
 * MOE_ERR_DEVICE_BAD_ID or MOE_ERR_DEVICE_TIMEOUT when a bit is set, else MOE_OK;
 * MOE_ERR_CUDA if the copy or the device lookup fails. Like the forward, it allocates
 * nothing; the word is shared by every caller of moe_forward_static on the device. */
moe_status moe_static_read_device_status(void* stream, int32_t* flags);

/* Router gate (vLLM MoE page, section "Gate 计算与 FSE"): router logits = x . wg^T with
 * fp32 accumulation, one GEMM for the routed experts' gate and, with n_shared = 1, the
 * fused shared-expert gate (FSE: wg is [E + 1, H], its last row the shared expert's gate).
 *   x              device bf16 [T, H]
 *   wg             device bf16 [E + n_shared, H]
 *   routed_logits  device fp32 [T, E]: the logits moe_route takes
 *   shared_logits  device fp32 [T] when n_shared = 1 (moe_forward_partial's shared_gate),
 *                  else ignored (may be NULL)
 * Requires H % 64 == 0 (64..32768), 1 <= E <= 256, n_shared in {0, 1}; 16-byte aligned
 * pointers. Deterministic: partial sums over K are added in a fixed order. */
moe_status moe_gate(const void* x, const void* wg, int64_t T, int32_t H, int32_t E,
                    int32_t n_shared, float* routed_logits, float* shared_logits, void* stream);

/* Router gate and routing in one launch (vLLM MoE page, section "Gate 计算与 FSE": the gate
 * GEMM that produces router_logits; TensorRT-LLM MoE page, layer-structure figure: fc_gate
 * ahead of routing): moe_gate, then moe_route on its logits. After the gate's fixed-order
 * reduction, the CTA that holds a token's complete row of routed logits routes the token
 * itself, so the logits need not travel through HBM to a second launch.
 *   x, wg, T, H, n_shared  as for moe_gate, with E = p->num_experts
 *   bias, p                as for moe_route (every method and envelope of moe_route)
 *   ids, scales            device int32 / fp32 [T, k] out, as moe_route writes them
 *   routed_logits          device fp32 [T, E] out, or NULL (then not written)
 *   shared_logits          device fp32 [T] out when n_shared = 1, else ignored (may be NULL)
 * The logits equal moe_gate's and the ids and scales equal moe_route's on those logits, bit
 * for bit. Errors: those of moe_gate and of moe_route, checked on the host before anything
 * is enqueued. */
moe_status moe_gate_route(const void* x, const void* wg, int64_t T, int32_t H, int32_t n_shared,
                          const float* bias, const moe_route_params* p, int32_t* ids,
                          float* scales, float* routed_logits, float* shared_logits,
                          void* stream);

/* moe_forward restricted to the experts [e_lo, e_hi) of this call: the expert-parallel
 * seam of the TensorRT-LLM MoE page, section on supports_finalize_before_combine ("finalize
 * before combine": the top-k weighted sum taken on a rank's own rows, slots of other
 * ranks' experts contributing exactly 0, so that the combine is an unweighted row sum).
 *   y[t] = sum over j with ids[t,j] in [e_lo, e_hi) of scales[t,j] * E_{ids[t,j]}(x[t])
 *          (+ shared(x[t]) when p->shared_I > 0)
 * The y of calls over a partition of [0, E) (the shared expert in exactly one of them) add
 * up to moe_forward's y. w13 / w2 hold the local experts only: [e_hi - e_lo, 2I, H] and
 * [e_hi - e_lo, H, I], expert g at plane g - e_lo. Requires 0 <= e_lo < e_hi <= E; ids in
 * [0, E) outside the range are not errors. shared_gate: device fp32 [T] logits of the
 * shared expert's gate (vLLM MoE page, "Gate 计算与 FSE": the shared expert's activation,
 * a sigmoid), so that it enters with weight sigmoid(shared_gate[t]); NULL = weight 1.
 * moe_forward is this call with [0, E) and no shared gate. */
moe_status moe_forward_partial(const moe_problem* p, int32_t e_lo, int32_t e_hi, const void* x,
                               const int32_t* ids, const float* scales, const void* w13,
                               const void* w2, const void* w13_s, const void* w2_s,
                               const float* shared_gate, void* y, void* workspace,
                               size_t ws_bytes, void* stream);

/* Step entry points (the kernels moe_forward runs, one at a time). Each takes the
 * same workspace; later steps read what earlier ones wrote into it. */

/* Step 2 (Dense GEMM -> GroupedGEMM article, sections 2.1-2.2: per-expert contiguous
 * blocks and an offset array). Clears the status word, then writes counts, starts,
 * offsets, the FC1/FC2 tile lists, perm_src, perm_inv and x_perm. Rows of an expert
 * keep ascending flat index f = t*k + j. */
moe_status moe_permute(const moe_problem* p, const void* x, const int32_t* ids,
                       void* workspace, size_t ws_bytes, void* stream);
/* Step 3: h[r, :] = silu(x_perm[r] . w13[e][0:I]^T) * (x_perm[r] . w13[e][I:2I]^T). */
moe_status moe_fc1(const moe_problem* p, const void* w13, const void* w13_s, void* workspace,
                   size_t ws_bytes, void* stream);
/* Step 4: out_perm[r, :] = h[r] . w2[e]^T. */
moe_status moe_fc2(const moe_problem* p, const void* w2, const void* w2_s, void* workspace,
                   size_t ws_bytes, void* stream);
/* Steps 3 and 4 as moe_forward runs them: one persistent launch whose work list holds
 * FC1's tiles, then FC2's; an FC2 tile starts once every FC1 tile of its expert has
 * stored its h rows (a per-expert completion counter in the workspace, bounded wait).
 * Same results, bit for bit, as moe_fc1 followed by moe_fc2. Call it after moe_permute on
 * the same workspace: that step zeroes the counters it uses. */
moe_status moe_fc1_fc2(const moe_problem* p, const void* w13, const void* w13_s, const void* w2,
                       const void* w2_s, void* workspace, size_t ws_bytes, void* stream);
/* Step 5 (TensorRT-LLM MoE page: routing weights applied after FC2; finalize = top-k
 * weighted row sum): y[t] = sum_j scales[t,j] * out_perm[perm_inv[t*k+j]] (+ shared row). */
moe_status moe_finalize(const moe_problem* p, const float* scales, void* y, void* workspace,
                        size_t ws_bytes, void* stream);

/* Synchronises `stream`, reads and clears the workspace status word. *flags (may be
 * NULL) receives the MOE_DEVICE_FLAG_* bits. Returns MOE_ERR_DEVICE_BAD_ID or
 * MOE_ERR_DEVICE_TIMEOUT when a bit is set, else MOE_OK. */
moe_status moe_read_device_status(void* workspace, void* stream, int32_t* flags);

/* Self-test of the device failure path, with no fault and no hang: one kernel (one CTA)
 * whose two pipeline roles wait on mbarriers that nothing arrives on, with the same
 * bounded wait as every pipelined kernel here (2 s of wall clock). The producer's wait
 * runs out, sets MOE_DEVICE_FLAG_TIMEOUT in the workspace status word and raises the
 * abort flag; the consumer, which started waiting 1 s later, leaves through that flag
 * and sets status word 1 to 1 when it left before its own limit. `workspace`: any
 * workspace of this library (16-byte aligned; only its first 16 bytes are touched, and
 * words 0-1 are cleared first). Enqueued on `stream`; returns at once. The timeout then
 * reads back through moe_read_device_status, and the context stays usable. Errors:
 * MOE_ERR_INVALID_ARG (NULL or misaligned workspace), MOE_ERR_CUDA (launch). */
moe_status moe_selftest_wait(void* workspace, void* stream);

/* Round-to-nearest-even conversion of n fp32 values to bf16 (device in/out). */
moe_status moe_cast_f32_to_bf16(const float* in, void* out, int64_t n, void* stream);

/* ---- Training operators: the layer's steps as calls of their own, on the caller's tensors, with
 * their gradients. They share nothing with the forward's workspace. All of them are
 * deterministic, enqueue on `stream` only and take contiguous row-major tensors that start on
 * 16-byte boundaries. A size outside the stated range returns MOE_ERR_UNSUPPORTED.
 *
 * T tokens, k slots a token (1..8), flat slot index f = t*k + j, E experts (1..256). */
typedef enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_F16 = 1, MOE_DTYPE_F32 = 2 } moe_dtype;

/* Rows of x [T, H] sorted by expert. ids [T, k]: the expert of each slot, or -1 for a slot that
 * was dropped. Slots are ordered by expert, then by f; dropped ones come last. place(f) is a
 * slot's row in that order:
 *   x_perm [T*k, H]   x_perm[place(f)] = x[f / k]; zeros in the rows of dropped slots
 *   inv [T, k]        place(f), or -1 - place(f) for a dropped slot
 *   offsets [E + 1]   the first row of each expert; offsets[E] = rows that are not dropped
 * dtype: any moe_dtype; H 1..65536; T <= 2^24. The workspace (moe_dispatch_workspace_bytes, 0
 * for sizes outside the range) needs no clearing; its status word, which
 * moe_read_device_status reads, gets MOE_DEVICE_FLAG_BAD_ID when an id is neither -1 nor in
 * [0, E) (the slot is then dropped). Up to MOE_DISPATCH_SMALL_SLOTS slots (T*k) need no workspace:
 * it may be NULL, and a bad id is then dropped without a flag. */
#define MOE_DISPATCH_SMALL_SLOTS 12288
size_t moe_dispatch_workspace_bytes(int64_t T, int32_t E, int32_t k);
moe_status moe_dispatch(const void* x, const int32_t* ids, int64_t T, int32_t H, int32_t E,
                        int32_t k, moe_dtype dtype, void* x_perm, int32_t* inv, int32_t* offsets,
                        void* workspace, size_t ws_bytes, void* stream);

/* x_perm alone, by an inv that is there already: for a backward pass that kept x, which is k
 * times smaller, in place of x_perm. In this and the next three calls a slot whose place lies
 * outside [0, T*k) counts as dropped and writes no row. */
moe_status moe_dispatch_rows(const void* x, const int32_t* inv, int64_t T, int32_t H, int32_t k,
                             moe_dtype dtype, void* x_perm, void* stream);

/* Gradient of moe_dispatch: dx[t] = sum over t's kept slots of dx_perm[inv[t, j]]. */
moe_status moe_dispatch_backward(const void* dx_perm, const int32_t* inv, int64_t T, int32_t H,
                                 int32_t k, moe_dtype dtype, void* dx, void* stream);

/* Back to token order: y[t] = sum over t's kept slots of scales[t, j] * rows[inv[t, j]], summed
 * in fp32 in slot order. scales [T, k] fp32, or NULL for 1. Rows of dropped slots are not read. */
moe_status moe_combine(const void* rows, const int32_t* inv, const float* scales, int64_t T,
                       int32_t H, int32_t k, moe_dtype dtype, void* y, void* stream);

/* Gradients of moe_combine: drows[place(f)] = scales[f] * dy[t] (zeros for a dropped slot) and
 * dscales[f] = <dy[t], rows[inv[f]]> (0 for a dropped slot). */
moe_status moe_combine_backward(const void* dy, const void* rows, const int32_t* inv,
                                const float* scales, int64_t T, int32_t H, int32_t k,
                                moe_dtype dtype, void* drows, float* dscales, void* stream);

/* SwiGLU that keeps its input for the backward pass in 8 bits. gu [R, 2I]: gate, then up, of each
 * row; h [R, I] = silu(gate) * up. The checkpoint is q [R, 2I], e4m3 values in gu's order, and
 * q_scales [R, 2 * ceil(I / 32)], a power of two 2^(byte - 127) for each 32 neighbouring channels
 * of the gate, then of the up half (the last of a half may cover fewer): the least with
 * |value| <= 448 * scale, so a value v is kept to within |v| / 16 (or 2^-10 of the scale). A
 * block that holds an infinity or a NaN has scale byte 255 and reads as NaN. dtype: any
 * moe_dtype; I 1..65536. */
moe_status moe_swiglu_ckpt(const void* gu, int64_t R, int32_t I, moe_dtype dtype, void* h,
                           uint8_t* q, uint8_t* q_scales, void* stream);

/* Its gradient at the kept values: dgu [R, 2I] from dh [R, I] and the checkpoint; and, where h is
 * not NULL, h [R, I] again, from the kept values, for the gradient of the weights behind it. */
moe_status moe_swiglu_ckpt_backward(const void* dh, const uint8_t* q, const uint8_t* q_scales,
                                    int64_t R, int32_t I, moe_dtype dtype, void* dgu, void* h,
                                    void* stream);

/* The experts' products over sorted rows: rows [offsets[e], offsets[e + 1]) are expert e's
 * (offsets [E + 1] int32 on the device, non-decreasing; the kernel keeps them inside [0, R] and in
 * order), w [E, N, K]. A part of the experts can be run with its part of a longer list of offsets.
 *   moe_experts_matmul      y [R, N]:     y[r] = x[r] . w[e]^T     (x [R, K])
 *   moe_experts_matmul_dx   dx [R, K]:    dx[r] = dy[r] . w[e]     (dy [R, N])
 *   moe_experts_matmul_dw   dw [E, N, K]: dw[e] = sum over e's rows of dy[r]^T . x[r]
 * Rows of no expert (before offsets[0], from offsets[E] on) are zeros in y and dx; an expert
 * without rows has dw = 0. fp32
 * accumulation, one rounding. dtype BF16 or F16; dw_dtype the same or F32, and with F32
 * `accumulate` adds to what dw holds. N and K: multiples of 8 up to 65536; R <= 2^23.
 * Workspace, 128-byte aligned, not cleared by the caller but for its status word (first 16 bytes):
 * for dw at least moe_experts_workspace_bytes(E) bytes (0 outside 1..256), status word cleared by
 * the call. The other two take NULL, or at least 16 bytes whose status word, cleared by the
 * caller once, receives MOE_DEVICE_FLAG_TIMEOUT (moe_read_device_status reads it). Given
 * moe_experts_split_bytes(product, ...) bytes, a product (0 forward, 1 dx, 2 dw) with few tiles
 * and a long contraction works on parts of it side by side; 0: this one does not. That changes
 * the order of the sums, not from run to run. */
size_t moe_experts_workspace_bytes(int32_t E);
size_t moe_experts_split_bytes(int32_t product, int64_t R, int32_t E, int32_t N, int32_t K);
moe_status moe_experts_matmul(const void* x, const void* w, const int32_t* offsets, int64_t R,
                              int32_t E, int32_t N, int32_t K, moe_dtype dtype, void* y,
                              void* workspace, size_t ws_bytes, void* stream);
moe_status moe_experts_matmul_dx(const void* dy, const void* w, const int32_t* offsets, int64_t R,
                                 int32_t E, int32_t N, int32_t K, moe_dtype dtype, void* dx,
                                 void* workspace, size_t ws_bytes, void* stream);
moe_status moe_experts_matmul_dw(const void* dy, const void* x, const int32_t* offsets, int64_t R,
                                 int32_t E, int32_t N, int32_t K, moe_dtype dtype,
                                 moe_dtype dw_dtype, int32_t accumulate, void* dw, void* workspace,
                                 size_t ws_bytes, void* stream);

/* Synchronises `stream`; reads and clears whether a bounded wait of the experts' products (above,
 * or on 4-bit operands), of the gate or of moe_layer_few ran out in any call on the current GPU,
 * with a workspace or without, since the last read. Such a call's results are incomplete. *flags
 * (may be NULL) receives MOE_DEVICE_FLAG_TIMEOUT or 0. Returns MOE_ERR_DEVICE_TIMEOUT when one did,
 * else MOE_OK. */
moe_status moe_read_timeouts(void* stream, int32_t* flags);

/* Self-test of that report, with no fault and no hang: one warp waits as the products do, without a
 * workspace, on a barrier that nothing arrives on, for the 2 s of every wait here. Enqueued on
 * `stream`; returns at once. */
moe_status moe_selftest_experts_wait(void* stream);

/* Gradient of moe_route's scales to its logits: dlogits [T, E] (every entry written) from logits
 * [T, E], the ids [T, k] that moe_route chose and dscales [T, k]. The choice itself has no
 * gradient (nor has the bias). Takes every method that moe_route runs; of the other parameters
 * only num_experts, top_k and routed_scaling_factor matter. Slots with an id outside [0, E) take
 * no part; non-finite logits count as -inf and get 0. */
moe_status moe_route_backward(const float* logits, const int32_t* ids, const float* dscales,
                              int64_t T, const moe_route_params* p, float* dlogits, void* stream);

/* ---- Serving with 4-bit operands --------------------------------------------------------
 *
 * Microscaled 4-bit floating point. A tensor [planes, rows, K] (a matrix: planes = 1) is held as
 *   codes   [planes, rows, K / 2] bytes: e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6; 8 is the sign), the lower
 *           channel in the low half of its byte
 *   scales  [planes, rows, S] bytes, S = K / block rounded up to a multiple of 16, one for each block of
 *           neighbouring channels; what fills a row up is written as 0 and not looked at
 *   MX      blocks of 32, byte b stands for 2^(b - 127), 255 for NaN
 *   NV      blocks of 16, an e4m3 number (0 or positive), times g: one f32 on the device for each plane,
 *           or NULL for 1
 * K: a multiple of 32 up to 65536. Tensors are 16-byte aligned, g 4-byte. */
typedef enum { MOE_FP4_MX = 0, MOE_FP4_NV = 1 } moe_fp4_format;

/* x [planes, rows, K] (any moe_dtype) to 4 bits. MX: the least power of two, 2^-127 or more, with every
 * |value| <= 6 * scale, so that nothing saturates. NV: the scale is amax / (6 g) rounded to nearest, 448
 * at most; a block whose scale rounds to 0 reads as zeros. Codes are value / scale (/ g) rounded to
 * nearest, 6 at most; ties to even everywhere; decided as on exact numbers. A block that holds an
 * infinity or a NaN gets the scale NaN and reads as NaN. g, positive and finite, is given (for weights,
 * say, amax / (6 * 448) of each expert, for rows a calibrated one); NULL with MX. planes * rows <= 2^31. */
moe_status moe_quantize_fp4(const void* x, int64_t planes, int64_t rows, int32_t K, moe_dtype dtype,
                            moe_fp4_format format, const float* g, uint8_t* codes, uint8_t* scales,
                            void* stream);
/* SwiGLU of gu [rows, 2I] (gate, then up) in fp32, its result [rows, I] held in 4 bits as above. */
moe_status moe_swiglu_fp4(const void* gu, int64_t rows, int32_t I, moe_dtype dtype,
                          moe_fp4_format format, const float* g, uint8_t* codes, uint8_t* scales,
                          void* stream);
/* The values again: out [planes, rows, K] of `dtype` (one past its range as an infinity). */
moe_status moe_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, const float* g,
                              int64_t planes, int64_t rows, int32_t K, moe_fp4_format format,
                              moe_dtype dtype, void* out, void* stream);

/* moe_experts_matmul with both operands in 4 bits of one format: y [R, N] (dtype BF16 or F16), y[r] =
 * x[r] . w[e]^T for the rows of expert e, x [R, K], w [E, N, K], x_g one value or NULL, w_g [E] or NULL.
 * Offsets, rows of no expert and limits as there (N a multiple of 8, K of 32). Products of codes and
 * scales are exact, their sums fp32, one rounding. */
moe_status moe_experts_matmul_fp4(const uint8_t* x_codes, const uint8_t* x_scales, const float* x_g,
                                  const uint8_t* w_codes, const uint8_t* w_scales, const float* w_g,
                                  const int32_t* offsets, int64_t R, int32_t E, int32_t N, int32_t K,
                                  moe_fp4_format format, moe_dtype dtype, void* y, void* stream);

/* The whole layer for a few tokens, in two kernels: moe_gate_route and moe_forward (with the shared
 * expert's gate, moe_forward_partial's) of T <= MOE_FEW_TOKENS tokens without the launches between them.
 * With 16-bit weights it takes less time than those two for a token or two, about as much for four; for more
 * it is the slower one unless there are many experts and H is 4096 or more.
 *   p        T, H, I, E, k and shared_I (0: no shared expert); H, I and shared_I multiples of 32, H up to
 *            32768, I and shared_I to 65536
 *   route    as moe_route takes it (DeepSeekV3 also with more than 32 experts a group), num_experts = E, top_k = k
 *   x [T, H], wg [E (+ 1), H] of `dtype` (BF16 or F16); shared_gate 1: wg's last row is the shared
 *            expert's gate, whose sigmoid is its weight, 0: weight 1
 *   w13 [E, 2I, H], w2 [E, H, I], w13_s [2 shared_I, H], w2_s [H, shared_I] (NULL without a shared expert)
 *            all of `dtype` (weights = MOE_WEIGHTS_16BIT), or all in 4 bits of one moe_fp4_format, g one
 *            f32 an expert (one for the shared expert's) or NULL
 * Writes y [T, H], ids int32 [T, k] and scales fp32 [T, k]. Between the products h, times its routing
 * weight, is rounded once: to bf16, or (f16 and 4-bit weights) to 11 bits beside its token's largest.
 * x and wg are not rounded (with 4-bit weights, what of x is less than 2^-29 of its token's largest is
 * rounded to steps of at most 2^-38 of that, an MX scale of 2^-127 counts as 0, and sums of MX products that
 * are less than 2^-90 and than 2^-105 of the token's largest lose bits), sums are fp32.
 * Experts that no token chose are not read. The results are the same on every run. Workspace:
 * moe_layer_few_workspace_bytes, 256-byte aligned, nothing of it has to be set; calls that share one
 * must be ordered. Whether a bounded wait ran out: moe_read_timeouts. */
#define MOE_FEW_TOKENS 16
#define MOE_WEIGHTS_16BIT (-1)
typedef struct {
  const void* w;          /* elements, or 4-bit codes */
  const uint8_t* scales;  /* of 4-bit weights, else NULL */
  const float* g;         /* of NV weights, or NULL */
} moe_weights;
/* 0 outside the limits. */
size_t moe_layer_few_workspace_bytes(const moe_problem* p);
moe_status moe_layer_few(const moe_problem* p, const moe_route_params* route, const void* x,
                         const void* wg, int32_t shared_gate, const float* bias, const moe_weights* w13,
                         const moe_weights* w2, const moe_weights* w13_s, const moe_weights* w2_s,
                         int32_t weights, moe_dtype dtype, int32_t* ids, float* scales, void* y,
                         void* workspace, size_t ws_bytes, void* stream);

/* moe_selftest_experts_wait of the products on 4-bit operands and of moe_layer_few: a wait as each has
 * them runs out after about 2 s and is reported by moe_read_timeouts, with no fault and no hang. */
moe_status moe_selftest_fp4_wait(void* stream);
moe_status moe_selftest_few_wait(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
