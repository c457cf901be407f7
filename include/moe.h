/*
 * libmoe — C ABI of the GB300 (sm_103a) MoE / MoD layer hot path.
 *
 * Sources, cited by page title and section:
 *   [FW] "PyTorch MoE/MoD Training Framework: custom CUDA kernels, DeepSpeed and
 *        7x speed-up on T4", section "What's in the box" (routing/gating =
 *        softmax over experts + top-k in one launch; dispatch and combine;
 *        sparse backward of gating and dispatch) and its Mixture-of-Depths
 *        paragraph (part of the tokens skips the layer).
 *   [EP] "Moonshot AI released MoonEP: Mixture-of-Experts training without GPU
 *        idle time", section "Step-by-step" (one contiguous [E(+B), H, H'] weight
 *        tensor per projection, experts addressed by row index; dispatch returns
 *        cu_seqlens) and section "What problem it solves" (maxvio skew; no
 *        per-layer CPU synchronisation).
 *   [T4] "MoE on T4: how to find and remove bottlenecks in training", table
 *        "RMSNorm, RoPE, SwiGLU" (SwiGLU = three matrix products).
 *
 * Conventions for every call:
 *   - Every pointer argument is a DEVICE pointer unless stated otherwise; the
 *     caller owns all memory.  The library never allocates, frees or
 *     synchronises (except moe_last_device_error, which synchronises `stream`).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Work is enqueued asynchronously on it.
 *   - Tensors are dense and row-major.  Activation/weight tensors use the
 *     storage type `dtype` (MOE_F32 = float, MOE_BF16 = bfloat16); router logits,
 *     gates, scores and their gradients are always float; indices are int32.
 *   - Every pointer must be 16-byte aligned (MOE_ERR_MISALIGNED otherwise) and
 *     the hidden size H must be a multiple of 8 (bf16) or 4 (fp32).
 *   - Argument errors are reported before anything is launched and nothing is
 *     written.  A CUDA launch error returns MOE_ERR_CUDA.  Kernels never trap:
 *     a device-side wait that exceeds its bound, or an index found out of range,
 *     sets a per-device error word that moe_last_device_error() returns.
 *   - Results are deterministic: the same inputs give bitwise-identical outputs.
 *   - T = tokens, H = hidden size, E = experts, K = experts per token,
 *     Hp = H' = expert FFN intermediate size, R = T*K routed rows.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,    /* bad size, null required pointer, bad enum */
  MOE_ERR_MISALIGNED = 2,     /* a pointer is not 16-byte aligned */
  MOE_ERR_WORKSPACE = 3,      /* workspace missing or smaller than moe_workspace_bytes() */
  MOE_ERR_UNSUPPORTED = 4,    /* valid but unsupported shape/dtype combination */
  MOE_ERR_CUDA = 5,           /* a CUDA runtime call or launch failed */
  MOE_ERR_TIMEOUT = 6,        /* device: a bounded wait gave up (reported by moe_last_device_error) */
  MOE_ERR_DEVICE_BOUNDS = 7   /* device: an index was out of range (reported by moe_last_device_error) */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

/* operation ids for moe_workspace_bytes */
enum { MOE_OP_ROUTE = 0, MOE_OP_DISPATCH = 1, MOE_OP_EXPERT_FFN = 2, MOE_OP_ROUTE_BWD = 3, MOE_OP_MOD_SELECT = 4,
       MOE_OP_EXPERT_FFN_BWD = 5, MOE_OP_COMBINE_NORM_BWD = 6, MOE_OP_EXPERT_FFN_W4 = 7, MOE_OP_ORTHOGONALIZE = 8,
       MOE_OP_MUON_STEP = 9 };

/* moe_gate modes: the score function, and bits that may be or-ed in */
enum { MOE_GATE_SOFTMAX = 0, MOE_GATE_SIGMOID = 1, MOE_GATE_RENORM = 0x10, MOE_GATE_GROUP_MAX = 0x20 };

/* moe_route_bwd modes; MOE_ROUTE_DX_WRITE may be or-ed in to overwrite dx instead
 * of accumulating into it, MOE_ROUTE_GATE_RENORM when the forward renormalised the
 * gates (moe_route_ex with MOE_ROUTE_RENORM) */
enum { MOE_ROUTE_SOFTMAX_TOPK = 0, MOE_ROUTE_MOD_LINEAR = 1, MOE_ROUTE_LOGIT_GRAD = 2,
       MOE_ROUTE_DX_WRITE = 0x100, MOE_ROUTE_GATE_RENORM = 0x200 };

/* moe_route_ex gate options (bit flags) */
enum { MOE_ROUTE_RENORM = 0x1, MOE_ROUTE_BIAS_SELECT = 0x2 };

/* Human-readable name of a status code (static string, never NULL). */
MOE_API const char* moe_status_str(int status);

/* ABI version (major*10000 + minor*100 + patch). */
MOE_API int moe_version(void);

/* Number of CUDA kernels this library has launched in this process (a host-side
 * counter; no device work).  Lets a caller count the launches of a region. */
MOE_API unsigned long long moe_kernel_launches(void);

/* Bytes of device workspace `op` needs for these sizes (0 = none; `ws` may then be
 * NULL).  Sizes not used by `op` are ignored.  Returns 0 for invalid sizes.
 * MOE_OP_EXPERT_FFN: the workspace is optional (see moe_expert_ffn). */
MOE_API size_t moe_workspace_bytes(int op, int T, int H, int E, int K, int Hp);

/* Synchronises `stream`, then returns and clears the current device's error word:
 * MOE_OK, MOE_ERR_TIMEOUT or MOE_ERR_DEVICE_BOUNDS (MOE_ERR_CUDA if the
 * synchronisation itself failed). */
MOE_API int moe_last_device_error(void* stream);

/* Diagnostic of the device-side failure detection.  Launches one kernel whose
 * single thread waits, with the same bounded wait every pipelined kernel of this
 * library uses, on a barrier that nothing ever arrives at.  After `wait_cycles` SM
 * clock cycles (1 .. 2^31) it gives up and records MOE_ERR_TIMEOUT in the device
 * error word, as a stalled copy or MMA pipeline would; nothing traps and the
 * context stays usable.  Returns the launch status (MOE_ERR_INVALID_ARG for
 * wait_cycles out of range); read the outcome with moe_last_device_error. */
MOE_API int moe_check_wait_timeout(unsigned long long wait_cycles, void* stream);

/*
 * Router: GEMM, softmax over experts and top-K gate       [FW "What's in the box"]
 *
 *   logits[t,e] = sum_h x[t,h] * w_router[h,e] + logit_bias[e]
 *   p[t,:]      = softmax(logits[t,:])
 *   topk_idx[t,:]  = the K experts with the largest logits, ordered by decreasing
 *                    logit, equal logits by increasing expert index
 *   topk_gate[t,k] = p[t, topk_idx[t,k]]   (no renormalisation after top-k)
 *
 *   x          [T,H]   dtype           w_router [H,E] dtype
 *   logit_bias [E]     float, nullable (added before softmax and selection)
 *   logits     [T,E]   float out (kept for moe_route_bwd)
 *   topk_idx   [T,K]   int32 out;  topk_gate [T,K] float out
 *   1 <= K <= E <= 1024, K <= 16.  bf16 needs E % 8 == 0.
 *   Workspace: moe_workspace_bytes(MOE_OP_ROUTE, T, H, E, K, 0) bytes (bf16 only):
 *   partial sums of the router GEMM over slices of H, added in a fixed order, for
 *   shapes whose token tiles alone would leave SMs idle; 0 (ws may be NULL) when the
 *   token tiles fill the GPU and for E = 8 or 16 with H a multiple of 512 up to 4096
 *   (those stream x through registers in one launch).  Results are the same bits on
 *   every run for the same inputs.
 */
MOE_API int moe_route(const void* x, const void* w_router, const float* logit_bias,
              int T, int H, int E, int K, int dtype,
              float* logits, int32_t* topk_idx, float* topk_gate,
              void* ws, size_t ws_bytes, void* stream);

/*
 * Router with gate options, for a drop-in replacement of a Mixtral-style sparse
 * MoE block                              [FW "How it looks in practice"]
 *
 * moe_route with `flags`, a bitwise or of
 *   MOE_ROUTE_RENORM       topk_gate[t,k] = p[t,topk_idx[t,k]] / sum_k' p[t,topk_idx[t,k']]
 *                          (the K gates of a token sum to 1, as in the Mixtral block);
 *   MOE_ROUTE_BIAS_SELECT  logit_bias shifts only the selection: topk_idx = the top K of
 *                          x w_router + logit_bias (same order and ties as above), while
 *                          logits, p and the gates are those of x w_router alone.
 * flags = 0 is exactly moe_route; other bits return MOE_ERR_INVALID_ARG.  Arguments,
 * layouts, workspace and errors as moe_route.  The backward of renormalised gates is
 * moe_route_bwd with MOE_ROUTE_GATE_RENORM; the selection-only bias needs no flag there
 * (the stored logits are unbiased).
 */
MOE_API int moe_route_ex(const void* x, const void* w_router, const float* logit_bias,
              int T, int H, int E, int K, int dtype, int flags,
              float* logits, int32_t* topk_idx, float* topk_gate,
              void* ws, size_t ws_bytes, void* stream);

/*
 * Gate with expert groups: scores, selection bias, group limit, top-K
 *
 *   s[t,e] = softmax(logits[t,:])[e]  (MOE_GATE_SOFTMAX)  or
 *            1 / (1 + exp(-logits[t,e]))  (MOE_GATE_SIGMOID)
 *   c[t,e] = s[t,e] + sel_bias[e]       (the bias shifts the selection only)
 *   The E experts form `groups` runs of E / groups neighbours.  A group ranks by the sum
 *   of its two largest c (by its largest with MOE_GATE_GROUP_MAX, or where it has one
 *   expert); the topk_groups highest stay, equal ranks by lower group.
 *   topk_idx[t,:]  = the K experts of those groups with the largest c, ordered by
 *                    decreasing c, equal c by increasing expert
 *   topk_gate[t,k] = scale * s[t,topk_idx[t,k]], with MOE_GATE_RENORM
 *                    scale * s[t,topk_idx[t,k]] / sum_k' s[t,topk_idx[t,k']]
 *
 *   The choice is that of scores in 64 bits: they are compared in fp32 where they are
 *   further apart than fp32's error and in fp64 where they are not (ranks that fp64's own
 *   rounding alone tells apart may go either way).  Without sel_bias the
 *   logits order as the scores do, and they are compared (but for the groups' sums).
 *   A logit of -inf takes an expert out of service: it ranks behind every expert in
 *   service (lower expert first), adds nothing to its group's rank (a group with one
 *   expert in service ranks by that one alone, one with none last), and its gate is 0,
 *   under MOE_GATE_RENORM too.  Scores too small for a float still have their quotients
 *   there: chosen logits that are all the type's lowest number have gates of scale / K.  A
 *   NaN logit, or a c that is NaN, ranks like -inf; a row that holds a NaN logit has NaN gates.
 *
 *   logits [T,E] float; sel_bias [E] float, nullable; topk_idx [T,K] int32 out;
 *   topk_gate [T,K] float out.  1 <= K <= E <= 1024, K <= 16, E a multiple of groups,
 *   1 <= topk_groups <= groups <= 32, topk_groups * (E / groups) >= K, scale finite.
 *   No workspace.
 */
MOE_API int moe_gate(const float* logits, const float* sel_bias, int T, int E, int K, int groups,
              int topk_groups, int mode, float scale, int32_t* topk_idx, float* topk_gate, void* stream);

/*
 * Router GEMM followed by moe_gate: logits = x w_router (kept for moe_gate_bwd), then the
 * gate above.  x, w_router, dtype, workspace and shape rules as moe_route; the rest as
 * moe_gate.  The gate reads the logits as stored, in fp32.
 */
MOE_API int moe_route_group(const void* x, const void* w_router, const float* sel_bias, int T, int H, int E,
              int K, int dtype, int groups, int topk_groups, int mode, float scale, float* logits,
              int32_t* topk_idx, float* topk_gate, void* ws, size_t ws_bytes, void* stream);

/*
 * Backward of moe_gate (no gradient through the selection; sel_bias has none)
 *
 *   with s, q = the chosen scores and the chosen scores rescaled to sum to 1:
 *   MOE_GATE_SIGMOID                  d_logits = scale * d_gate * s (1 - s) at the chosen experts
 *   MOE_GATE_SIGMOID|MOE_GATE_RENORM  d_logits = scale * q (1 - s) (d_gate - <d_gate, q>)
 *   MOE_GATE_SOFTMAX                  d_logits = scale * s (G - <d_gate, s>) over the whole row,
 *                                     G = d_gate at the chosen experts, 0 elsewhere
 *   MOE_GATE_SOFTMAX|MOE_GATE_RENORM  d_logits = scale * q (d_gate - <d_gate, q>)
 *   and 0 elsewhere; an expert listed twice in a row receives the sum of its shares.  A NaN logit shows in
 *   what the formula makes of it: the whole row, or the chosen experts, or its own place alone.
 *   d_gate [T,K], logits [T,E] float; topk_idx [T,K] int32 as moe_gate wrote it (an index
 *   outside [0,E) sets MOE_ERR_DEVICE_BOUNDS and has no share); d_logits [T,E] float out,
 *   apart from logits, every element written.  MOE_GATE_GROUP_MAX is accepted and changes nothing.  Sizes as
 *   moe_gate.  dw_router and dx follow with moe_route_bwd(MOE_ROUTE_LOGIT_GRAD).
 */
MOE_API int moe_gate_bwd(const float* d_gate, const float* logits, const int32_t* topk_idx, int T, int E, int K,
              int mode, float scale, float* d_logits, void* stream);

/*
 * Dispatch: expert histogram, prefix sum, permutation, gather
 *                              [FW "What's in the box"; EP "Step-by-step"]
 *
 *   cu_seqlens[0] = 0, cu_seqlens[e+1] = cu_seqlens[e] + #{(t,k): topk_idx[t,k] = e},
 *   so cu_seqlens[E] = T*K.  Rows of expert e are [cu_seqlens[e], cu_seqlens[e+1])
 *   of one contiguous expert-sorted buffer, in increasing token order (stable).
 *   dst_row[t*K+k] = row of pair (t,k);  src_tok[row] = t;  xs[row,:] = x[t,:].
 *
 *   x [T,H] dtype; topk_idx [T,K] int32 with distinct experts per token in [0,E)
 *   cu_seqlens [E+1], dst_row [T*K], src_tok [T*K] int32 out; xs [T*K,H] dtype out,
 *   nullable: without xs only the index maps are written (x may then be NULL)
 *   and moe_expert_ffn_gather reads the rows of x itself.
 *   An expert id outside [0,E) sets MOE_ERR_DEVICE_BOUNDS; its pair is dropped.
 *   Workspace: moe_workspace_bytes(MOE_OP_DISPATCH, T, 0, E, K, 0) bytes.
 */
MOE_API int moe_dispatch(const void* x, const int32_t* topk_idx, int T, int H, int E, int K, int dtype,
                 int32_t* cu_seqlens, int32_t* dst_row, int32_t* src_tok, void* xs,
                 void* ws, size_t ws_bytes, void* stream);

/*
 * moe_dispatch without a workspace argument.  The source pages have no
 * counterpart for this call; it exists for callers that cannot allocate device
 * memory: code whose device memory is owned by someone else (a framework
 * allocator or a fixed arena planned ahead of time) and that has no scratch
 * buffer to hand over, or code that must not call cudaMalloc on its hot path,
 * where it can synchronise the device or fail under memory pressure.
 *
 * Same arguments, results and errors as moe_dispatch, minus ws/ws_bytes.  The
 * scratch it needs (a ceil(T/256) x E table of int32 counts and E int32 totals)
 * is a library-owned static device array of 65536 ints (256 KB), present on
 * every GPU that loads the library until the process exits.  Sizes with
 * ceil(T/256) * E + E > 65536 return MOE_ERR_WORKSPACE before anything is
 * launched.  The call allocates
 * nothing (no cudaMalloc/cudaFree, no allocating library routine).
 *
 * The first call on a device looks up the array's device address (one
 * cudaGetSymbolAddress with that device current); make that first call before
 * any stream capture.  Every call shares the one array: nothing in it needs
 * clearing between calls, but calls whose kernels may overlap on the GPU (e.g.
 * on two streams with no ordering between them) race and must be serialised
 * by the caller.
 */
MOE_API int moe_dispatch_noalloc(const void* x, const int32_t* topk_idx, int T, int H, int E, int K,
                                 int dtype, int32_t* cu_seqlens, int32_t* dst_row, int32_t* src_tok,
                                 void* xs, void* stream);

/*
 * Grouped SwiGLU expert FFN over contiguous weights
 *                [EP "Step-by-step" (weights [E,H,H'], rows by index); T4 SwiGLU]
 *
 *   For every expert e and row r in [cu_seqlens[e], cu_seqlens[e+1]):
 *     act[r,:] = silu(xs[r,:] . w_gate[e]) * (xs[r,:] . w_up[e])     silu(z) = z/(1+exp(-z))
 *     h[r,:]   = act[r,:] . w_down[e]^T
 *   xs [rows,H]; w_gate, w_up, w_down each one contiguous [E,H,Hp] tensor (dtype);
 *   act [rows,Hp] and h [rows,H] dtype out.  Accumulation is fp32; bf16 outputs
 *   are rounded to nearest-even (silu in fp32 with exp and divide of a few ulp;
 *   moe_expert_ffn_ex with gu divides exactly, so its act may differ from this
 *   call's in the last bit).  The row split is read on the device from
 *   cu_seqlens (no host synchronisation); cu_seqlens[E] must equal `rows`.
 *   bf16 needs H % 64 == 0 and Hp % 64 == 0.
 *   Workspace (optional, bf16): with ws 16-byte aligned and ws_bytes >=
 *   moe_workspace_bytes(MOE_OP_EXPERT_FFN, ...) (about 32 MB, independent of the
 *   sizes), when the down projection's last round of 256 x 256 tiles holds at
 *   most half as many tiles as the GPU runs CTA pairs, each of those tiles is
 *   computed as two K halves on two pairs whose fp32 partials are added (once,
 *   in fp32) before the bf16 rounding; the workspace holds the partials and
 *   arrival counters (the gate/up kernel of the same call zeroes them; no
 *   state carries between calls).  h then differs from a call without the
 *   workspace by that one extra fp32 rounding in those tiles; for the same
 *   inputs on the same GPU model it is deterministic.  NULL or fewer bytes:
 *   whole tiles only.  Concurrent calls need distinct workspaces.
 */
MOE_API int moe_expert_ffn(const void* xs, const int32_t* cu_seqlens, int rows,
                   const void* w_gate, const void* w_up, const void* w_down,
                   int E, int H, int Hp, int dtype, void* act, void* h,
                   void* ws, size_t ws_bytes, void* stream);

/*
 * Grouped SwiGLU expert FFN with the dispatch gather fused into its input load
 *                      [FW "What's in the box": dispatch reads the buffers
 *                       directly; EP "Step-by-step": rows addressed by index]
 *
 *   moe_expert_ffn_ex with xs[r,:] = x[src_tok[r],:] read straight from x: in
 *   the gate/up GEMM (CTA pairs, 256-row tiles) eight extra warps per CTA copy
 *   the CTA's 128 rows of each tile from x by src_tok (as written by
 *   moe_dispatch) into its operand stages, so the expert-sorted copy of the
 *   input is never written or read.  The results are bit-identical to
 *   moe_expert_ffn_ex on the rows moe_dispatch writes (with the same
 *   workspace argument).  x [T,H] dtype; src_tok [rows] int32 in [0,T) (an
 *   index outside sets MOE_ERR_DEVICE_BOUNDS and reads row 0); the rest as
 *   moe_expert_ffn_ex.
 *   Workspace: optional, as moe_expert_ffn (the down projection's tail split).
 */
MOE_API int moe_expert_ffn_gather(const void* x, const int32_t* src_tok, int T, const int32_t* cu_seqlens,
                                  int rows, const void* w_gate, const void* w_up, const void* w_down, int E,
                                  int H, int Hp, int dtype, void* act, void* gu, void* h, void* ws,
                                  size_t ws_bytes, void* stream);

/*
 * Expert FFN forward that also keeps the SwiGLU pre-activations for the backward
 *
 * moe_expert_ffn plus gu [rows, 2*Hp] dtype out (nullable): gu[r, 0:Hp] = g =
 * xs[r,:] . w_gate[e] and gu[r, Hp:2Hp] = u = xs[r,:] . w_up[e], rounded to dtype.
 * gu needs bf16 (MOE_ERR_UNSUPPORTED otherwise).  gu = NULL is moe_expert_ffn.
 */
MOE_API int moe_expert_ffn_ex(const void* xs, const int32_t* cu_seqlens, int rows,
                   const void* w_gate, const void* w_up, const void* w_down,
                   int E, int H, int Hp, int dtype, void* act, void* gu, void* h,
                   void* ws, size_t ws_bytes, void* stream);

/*
 * Expert FFN backward         [T4 "RMSNorm, RoPE, SwiGLU": SwiGLU = three matrix
 *                              products; FW "What's in the box": the layer trains]
 *
 * Given dh = dL/dh [rows,H] for the forward above (gu and act as the forward wrote
 * them), for every expert e and its rows:
 *   da  = dh . w_down[e]                        [rows_e, Hp]
 *   dg  = da * u * s(g) * (1 + g (1 - s(g)))    du = da * g * s(g)      s = logistic
 *   dxs = dg . w_gate[e]^T + du . w_up[e]^T     [rows_e, H]   dtype out (nullable)
 *   dw_gate[e] = xs_e^T dg,  dw_up[e] = xs_e^T du,  dw_down[e] = dh_e^T act_e
 *                                               [E,H,Hp] float out each (nullable);
 *                                               zero for experts without rows
 * bf16 only (MOE_ERR_UNSUPPORTED otherwise), same shape rules as moe_expert_ffn.
 * Workspace: moe_workspace_bytes(MOE_OP_EXPERT_FFN_BWD, T, H, E, K, Hp) bytes with
 * T*K = rows (it holds [dg | du], bf16).  Weight gradients are written, not
 * accumulated, each element reduced over its expert's rows in one fp32 accumulator.
 */
MOE_API int moe_expert_ffn_bwd(const void* xs, const int32_t* cu_seqlens, int rows,
                   const void* w_gate, const void* w_up, const void* w_down,
                   int E, int H, int Hp, int dtype, const void* gu, const void* act, const void* dh,
                   void* dxs, float* dw_gate, float* dw_up, float* dw_down,
                   void* ws, size_t ws_bytes, void* stream);

/*
 * Combine: gate-weighted sum back to token order        [FW "What's in the box"]
 *
 *   y[o(t),:] = residual[o(t),:] + s_t * sum_k gate[t,k] * h[dst_row[t*K+k],:]
 *   o(t) = out_row[t] (nullable: o(t) = t);  s_t = row_scale[t] (nullable: 1);
 *   residual nullable (then 0), indexed like y.  Accumulated in fp32 in k order.
 *   dst_row nullable: then dst_row[j] = j.
 *   h [T*K,H] dtype; gate [T,K] float; y dtype out; only rows o(t) are written.
 */
MOE_API int moe_combine(const void* h, const float* gate, const int32_t* dst_row,
                const float* row_scale, const void* residual, const int32_t* out_row,
                int T, int H, int K, int dtype, void* y, void* stream);

/*
 * Router backward                         [FW "What's in the box", sparse backward]
 *
 * mode MOE_ROUTE_SOFTMAX_TOPK (gate[t,k] = softmax(logits[t])[topk_idx[t,k]]):
 *   d_logits[t,j] = p_j * (G_j - sum_k d_gate[t,k] * p[topk_idx[t,k]]),
 *                   G_j = d_gate[t,k] if j = topk_idx[t,k] else 0  (no gradient
 *                   through the selection itself)
 *   dw_router[h,e] = sum_t x[t,h] * d_logits[t,e]      (float, nullable)
 *   dx[t,h]       += sum_e d_logits[t,e] * w_router[h,e] (dtype, nullable, accumulated;
 *                   written instead when mode has MOE_ROUTE_DX_WRITE)
 * with MOE_ROUTE_GATE_RENORM or-ed in (gate[t,k] = q_k = p[topk_idx[t,k]] / sum_k' p[topk_idx[t,k']]):
 *   d_logits[t,topk_idx[t,k]] = q_k * (d_gate[t,k] - sum_k' d_gate[t,k'] * q_k'), 0 elsewhere
 * mode MOE_ROUTE_MOD_LINEAR (scalar score s[t] = x[t] . w; pass E = K = 1,
 *   w_router = w [H], d_gate = d_score [T], logits/topk_idx unused):
 *   d_logits = d_score (nullable), dw_router[h] = sum_t d_score[t] x[t,h],
 *   dx[t,h] += d_score[t] * w[h].
 * mode MOE_ROUTE_LOGIT_GRAD (d_gate holds the logit gradient [T,E] itself, e.g. from
 *   moe_gate_bwd; E % 4 == 0; logits and topk_idx unused, d_logits NULL): dw_router and dx as above.
 * The weight gradient is reduced deterministically through the workspace:
 *   moe_workspace_bytes(MOE_OP_ROUTE_BWD, T, H, E, K, 0) bytes.
 */
MOE_API int moe_route_bwd(int mode, const float* d_gate, const float* logits, const int32_t* topk_idx,
                  const void* x, const void* w_router, int T, int H, int E, int K, int dtype,
                  float* d_logits, float* dw_router, void* dx,
                  void* ws, size_t ws_bytes, void* stream);

/*
 * Backward of combine (and of the dispatch gather)  [FW "What's in the box"]
 *
 * With g(t) = dy[o(t)] (o, s_t as in moe_combine):
 *   dh[dst_row[t*K+k]] = s_t * gate[t,k] * g(t)                 (dtype, nullable)
 *   d_gate[t,k]        = s_t * <g(t), h[dst_row[t*K+k]]>        (float, nullable)
 *   d_scale[t]         = sum_k gate[t,k] * <g(t), h[dst_row[t*K+k]]> (float, nullable)
 *   dx[t]              = sum_k dxs[dst_row[t*K+k]]              (dtype, written; nullable,
 *                                                                requires dxs)
 * Dot products and sums accumulate in fp32.
 */
MOE_API int moe_permute_bwd(const void* dy, const void* h, const float* gate, const int32_t* dst_row,
                    const float* row_scale, const int32_t* out_row, const void* dxs,
                    int T, int H, int K, int dtype,
                    void* dh, float* d_gate, float* d_scale, void* dx, void* stream);

/*
 * Combine fused with the norms around the block, its gate and its residual scale
 *
 *   z[t,:]  = sum_k gate[t,k] * h[dst_row[t*K+k],:]
 *   n[t,:]  = z[t,:] / sqrt(mean(z[t,:]^2) + eps) * w_post      (w_post NULL: n = z)
 *   y[t,:]  = residual[t,:] + row_scale[t] * res_scale[:] * n[t,:]
 *   xn[t,:] = y[t,:] / sqrt(mean(y[t,:]^2) + eps) * w_next      (w_next NULL: no xn)
 *
 *   One pass: the block's output never returns to memory, and xn is computed from y before
 *   y is rounded to dtype.  Sums and means are fp32.
 *   h [T*K,H] dtype, nullable: without it y = residual, and only xn is written (the norm
 *   before the first block); gate, dst_row, row_scale, w_post, res_scale and y must then be
 *   NULL and K 0.
 *   gate [T,K] float, nullable (1); dst_row [T*K] int32 in [0,T*K), nullable (t*K+k; an
 *   index outside sets MOE_ERR_DEVICE_BOUNDS and counts as a row of zeros);
 *   row_scale [T] float, nullable (1); residual [T,H] dtype, nullable (0; required without
 *   h); w_post, res_scale, w_next [H] float, nullable; y, xn [T,H] dtype out.  y may be
 *   the same buffer as residual; no other overlap.  eps > 0, finite.  1 <= K <= 16 with h;
 *   H <= 16384.  No workspace.
 */
MOE_API int moe_combine_norm(const void* h, const float* gate, const int32_t* dst_row, const float* row_scale,
              const void* residual, const float* w_post, const float* res_scale, const float* w_next, float eps,
              int T, int H, int K, int dtype, void* y, void* xn, void* stream);

/*
 * Backward of moe_combine_norm
 *
 *   dy, dxn = dL/dy and dL/dxn of the forward above, y as it stored it (its norm's
 *   statistics and the block's are recomputed: nothing else is kept).  With
 *   v = y / sqrt(mean(y^2) + eps), r = 1 / sqrt(mean(z^2) + eps), u = r z (u = z without w_post),
 *   a missing w_post, res_scale or row_scale read as 1:
 *     D        = dy + (w_next dxn - v mean(w_next dxn v)) / sqrt(mean(y^2) + eps)
 *     d_res    = D
 *     P        = row_scale res_scale w_post D
 *     dz       = r (P - u mean(P u))                (dz = P without w_post)
 *     dh[dst_row[t*K+k],:] = gate[t,k] dz[t,:];  d_gate[t,k] = <dz[t,:], h[dst_row[t*K+k],:]>
 *     d_scale[t] = sum_c D res_scale w_post u
 *     dw_post = sum_t row_scale res_scale D u;  d_res_scale = sum_t row_scale w_post D u
 *     dw_next = sum_t dxn v
 *   dy [T,H] dtype, nullable (0) where dxn is given; dxn and w_next both or neither, and y
 *   with them (otherwise y is unused).  h, gate, dst_row, row_scale, w_post, res_scale, eps,
 *   T, H, K, dtype as in the forward (h NULL: the norm alone).
 *   Outputs, each nullable: d_res [T,H], dh [T*K,H] dtype (dst_row a permutation);
 *   d_gate [T,K], d_scale [T] float; dw_post (needs w_post), d_res_scale (needs res_scale),
 *   dw_next (needs w_next) [H] float, written, not accumulated.  d_res may be the same
 *   buffer as dy or dxn; no other overlap.
 *   Workspace: moe_workspace_bytes(MOE_OP_COMBINE_NORM_BWD, T, H, 0, K, 0) bytes (partial
 *   column sums, added in a fixed order); it may be NULL where the three column sums are.
 *   Calls that may run at the same time need distinct workspaces.
 */
MOE_API int moe_combine_norm_bwd(const void* dy, const void* dxn, const void* h, const float* gate,
              const int32_t* dst_row, const float* row_scale, const void* y, const float* w_post,
              const float* res_scale, const float* w_next, float eps, int T, int H, int K, int dtype,
              void* d_res, void* dh, float* d_gate, float* d_scale, float* dw_post, float* d_res_scale,
              float* dw_next, void* ws, size_t ws_bytes, void* stream);

/*
 * Activation checkpoint in 8 bits
 *
 *   Every run of 32 neighbours of a row (the last one of a row may be shorter) shares one
 *   power of two: with a = max |x| of the run, e = the least integer >= -126 with
 *   a <= 127 * 2^e, scale[row, run] = e + 127, q = x / 2^e rounded to the nearest integer,
 *   halves to even.  A value is off by at most 2^(e-1): where a > 127 * 2^-127, so that e follows
 *   a, at most a / 127 (a / 254 to a / 127 by where a lies between powers of two); in smaller
 *   runs 2^-127, whatever a.  A run that holds an infinity or a NaN has scale 255 and q 0, and is
 *   restored as NaN.
 *   x [rows,N] dtype; q [rows,N] int8 out; scale [rows, ceil(N/32)] uint8 out.  N a
 *   multiple of 8 (bf16) or 4 (fp32), at most 2^31 - 32.
 */
MOE_API int moe_ckpt_pack(const void* x, int rows, int N, int dtype, int8_t* q, uint8_t* scale, void* stream);

/* x[row, c] = q[row, c] * 2^(scale - 127): what the checkpoint stands for (exact in both types
 * unless the power of two falls below the type's range). */
MOE_API int moe_ckpt_unpack(const int8_t* q, const uint8_t* scale, int rows, int N, int dtype, void* x, void* stream);

/*
 * The checkpoint of [g | u] in the expert FFN's backward
 *
 *   q [rows, 2*Hp], scale [rows, ceil(2*Hp/32)] = moe_ckpt_pack of the gu that
 *   moe_expert_ffn_ex wrote.  gu [rows, 2*Hp] dtype out (nullable) = the restored g and u;
 *   act [rows, Hp] dtype out (nullable) = silu(g) * u of the restored values: the two inputs
 *   that moe_expert_ffn_bwd takes from the forward.  Hp a multiple of 8 (bf16) or 4 (fp32).
 */
MOE_API int moe_ckpt_swiglu(const int8_t* q, const uint8_t* scale, int rows, int Hp, int dtype, void* gu, void* act,
              void* stream);

/*
 * Expert weights in 4 bits with group scales
 *
 *   w [E, rows, cols] dtype, one of the expert tensors.  `axis` is the one that its product
 *   sums over: 0 (rows; w_gate and w_up, [E, H, H']) or 1 (cols; w_down).  With in = the size
 *   of that axis, out = the other one's, and B = ceil(in / 128) blocks:
 *     every `group` (32, 64 or 128) neighbours along `axis` of one output share a scale;
 *     with a = max |w| of the group, s = the least number of 5 significant bits >= a * (1 / 7) (both
 *     rounded to fp32), at least 2^-126.  Where a is 7 times a lower such number, as 1 / 7 in fp32 is above 1/7, and
 *     every weight of the group is a whole multiple of it, s is that number: what moe_w4_unpack restored of a tensor
 *     packed here (of magnitudes below 2^126) packs to the same codes and scales.  code = w / s (in fp32) rounded to the nearest
 *     integer, halves to even: -7..7.  code * s has at most 8 significant bits and is exact in
 *     bf16.  A value is off by at most s / 2 (1 + 2^-20), and s <= 17/16 * a / 7 * (1 + 2^-20) where that
 *     is above 2^-126.
 *     A group that holds a NaN, an infinity or a magnitude of 2^127 or more has the scale NaN
 *     and is restored as NaN.
 *   q     [E, out, B * 16] 32-bit words, 8 codes (as code + 8) in each: inputs 128 b + 32 j + 8 v
 *         .. + 7 (0 <= j, v < 4) are word 16 b + 4 v + j, input i of them in bits 4 (i / 2) + 16 (i % 2)
 *   scale [E, out, B * 128 / group] bf16
 *   Inputs past `in` (the last block's rest) are written as zeros.  E * rows * cols may pass
 *   2^31.  rows and cols multiples of 8 (bf16) or 4 (fp32), at most 2^23; E <= 65535.  q and scale
 *   of tensors made elsewhere may hold any codes (-8 too) and any bf16 scales below 2^125 in
 *   magnitude (whose 8-fold is finite): where a scale has more than 5 significant bits, code * s is
 *   rounded to bf16 by moe_w4_unpack to bf16, and by moe_expert_ffn_w4 but in its form for the fewest rows.
 */
MOE_API int moe_w4_pack(const void* w, int E, int rows, int cols, int axis, int group, int dtype, uint32_t* q,
              void* scale, void* stream);

/* w = code * s: the weights that the packed form stands for (arguments as moe_w4_pack). */
MOE_API int moe_w4_unpack(const uint32_t* q, const void* scale, int E, int rows, int cols, int axis, int group, int dtype,
              void* w, void* stream);

/*
 * Expert FFN with weights of 4 bits
 *
 *   act[r,:] = silu(xs[r,:] Wg[e]) * (xs[r,:] Wu[e]),  h[r,:] = act[r,:] Wd[e]^T
 *   for row r of expert e, as moe_expert_ffn, with the three tensors as moe_w4_pack makes them:
 *   q_gate, s_gate and q_up, s_up of [E,H,Hp] with axis 0, q_down, s_down of [E,H,Hp] with axis 1,
 *   all with the same `group`.
 *   x, src_tok: the routed rows, as in moe_expert_ffn_gather (row r reads x[src_tok[r],:], x [T,H]);
 *   src_tok NULL: x is xs [rows,H], as in moe_expert_ffn, and T is not used.  An entry of src_tok
 *   outside [0,T) sets MOE_ERR_DEVICE_BOUNDS and counts as a row of zeros.  So does a cu_seqlens that
 *   does not run from 0 to rows: offsets outside are read as if cut off there, and with one below the one before
 *   it nothing is computed.  Rows of no expert are left as they are.
 *   act [rows,Hp], h [rows,H] dtype out.  Products are fp32 sums of bf16 rows and exact weights; act
 *   is rounded to dtype before the second product.  For serving, from one row to a few hundred an
 *   expert: the weights are read in 4 bits once for each 8 to 128 rows of an expert.
 *   dtype MOE_BF16; H and Hp multiples of 8, at most 2^20; E <= 1024.  Workspace:
 *   moe_workspace_bytes(MOE_OP_EXPERT_FFN_W4, T, H, E, K, Hp) bytes for rows = T * K, with src_tok alone
 *   (without it, or where it is 0: NULL).  Calls that may run at the same time need distinct
 *   workspaces.  act and h overlap no other tensor of the call.
 */
MOE_API int moe_expert_ffn_w4(const void* x, const int32_t* src_tok, int T, const int32_t* cu_seqlens, int rows,
              const uint32_t* q_gate, const void* s_gate, const uint32_t* q_up, const void* s_up, const uint32_t* q_down,
              const void* s_down, int E, int H, int Hp, int group, int dtype, void* act, void* h, void* ws,
              size_t ws_bytes, void* stream);

/*
 * Orthogonalised matrices by Newton-Schulz products
 *
 *   For each of E matrices U = x[e] [M,N]:  X = U / (|U|_F + eps), then `steps` times
 *     X <- a X + b (X X^T) X + c (X X^T)^2 X
 *   (computed on the shorter side).  With the Muon optimiser's coefficients (3.4445, -4.7750,
 *   2.0315) and 5 steps the singular values that are not far below the largest come to about 1.
 *   x [E,M,N] dtype; out [E,M,N] bf16 (dtype names x's type).  out may not overlap x.
 *   The products' operands are fp16 (2^10 times X, which is below 2 there for such coefficients)
 *   with fp32 sums, the diagonals of X X^T and of the polynomial fp32: for matrices of noise with
 *   some directions that stand out the result is within about 2e-3 of exact arithmetic (2-norm, relative).
 *   What is far below x's root mean square singular value (some 2^-11 of it) is not resolved: such
 *   directions come out small, not as in exact arithmetic.  Where they are most of them, that is the larger error: the
 *   rounding of X puts noise into the empty directions of a matrix of low rank r (the gradient of an expert that had r
 *   rows), and five steps with these coefficients make it up to 3.4445^5 = 485 times larger: 0.1 to 0.15 in the Frobenius
 *   norm at any size, where the result has about sqrt(r).  Relative to it 0.15 for r = 1, 0.04 for 8, 0.02 for 64.
 *   With coefficients that let an element of X, of X X^T off its diagonal or of the polynomial off its own pass 63 on the way,
 *   that element is infinite.
 *   The norm neither over- nor underflows.  A matrix of zeros gives zeros; one that holds a NaN or
 *   an infinity gives NaN; the others of the batch are not touched by it.
 *   1 <= steps <= 64; a, b, c finite; eps >= 0, finite; 1 <= M, N <= 65536; E <= 65535.  Any M and N.
 *   Workspace: moe_workspace_bytes(MOE_OP_ORTHOGONALIZE, 0, M, E, 0, N) bytes.  With m = min(M, N) and n = max(M, N),
 *   both rounded up to 64 where they count columns: 4 m (n + m) + 8 m + 6152 bytes a matrix (4 to 8 for each element of large
 *   ones), and where up to 25 tiles of 256 x 256 of X X^T are too few for the GPU and n is long, one fp32 tile for
 *   each of up to 76 parts (20 MB).  It is asked for at every size.  Calls that may run at the same time need distinct
 *   workspaces.
 */
MOE_API int moe_orthogonalize(const void* x, int E, int M, int N, int dtype, int steps, float a, float b, float c,
              float eps, void* out, void* ws, size_t ws_bytes, void* stream);

/*
 * Momentum step with an orthogonalised update, on an expert tensor
 *
 *   m_out = beta m + dw
 *   u     = m_out, or with nesterov dw + beta m_out
 *   O     = moe_orthogonalize of u (steps, a, b, c, eps), not rounded
 *   w_out = (1 - lr weight_decay) w - lr scale O
 *   w, w_out [E,M,N] dtype; dw, m, m_out [E,M,N] float (dw as moe_expert_ffn_bwd writes it);
 *   w_low [E,M,N] bf16, nullable: w_out rounded to bf16 (with dtype MOE_F32, for weights kept in
 *   fp32 that the products read in bf16).  w_out may be w, m_out may be m; no other overlap.
 *   0 <= beta < 1; lr, weight_decay, scale finite; nesterov 0 or 1; the rest, the workspace
 *   (MOE_OP_MUON_STEP) and the accuracy of O as moe_orthogonalize.  Sums are fp32.
 */
MOE_API int moe_muon_step(const void* w, const float* dw, const float* m, int E, int M, int N, int dtype, float beta,
              int nesterov, float lr, float weight_decay, float scale, int steps, float a, float b, float c, float eps,
              void* w_out, void* w_low, float* m_out, void* ws, size_t ws_bytes, void* stream);

/*
 * Mixture-of-Depths capacity router                       [FW, MoD paragraph]
 *
 *   score[b*L+i] = x[b*L+i,:] . w_mod                              (float out)
 *   per sequence b: the C positions with the highest score (equal scores -> lower
 *   position) are selected; sel[b*C+j] = the j-th selected position, ascending
 *   as a flat token index b*L + position (int32 out); mask[b*L+i] = 1 if selected
 *   (u8 out).
 *   Optional outputs (nullable):
 *     sel_score[b*C+j] = score of that token (float)  -> row_scale of moe_combine
 *     x_sel[b*C+j,:]   = x[sel[b*C+j],:]               -> input of the MoE
 *     y_skip: y[b*L+i,:] = x[b*L+i,:] for every unselected token (the skip path)
 *   x [B*L,H], w_mod [H] dtype.  1 <= L <= 8192, 0 <= C <= L.  Workspace: none.
 */
MOE_API int mod_select(const void* x, const void* w_mod, int B, int L, int H, int C, int dtype,
               float* score, int32_t* sel, float* sel_score, uint8_t* mask,
               void* x_sel, void* y_skip, void* ws, size_t ws_bytes, void* stream);

/*
 * Expert-parallel dispatch plan (host only)      [EP "Step-by-step": the S x K
 *                      rows per rank invariant, the preload pool of B slots,
 *                      the [E+B, H, H'] weights addressed by row index]
 *
 *   R ranks, E experts (E % R == 0; rank r owns experts [rG, rG+G), G = E/R),
 *   S tokens per rank, K experts per token, B preload slots per rank.
 *   counts [R][E] int32: pairs that source rank s routes to expert e; every row
 *   must sum to S*K (MOE_ERR_INVALID_ARG otherwise).
 *   Outputs (caller-owned host arrays):
 *     piece_count [R][R][E], piece_offset [R][R][E]: destination rank d
 *       processes pairs [offset, offset + count) of source s's pairs for expert
 *       e (in the source's (t, k) order);
 *     slot_expert [R][B]: the expert whose weights slot j of rank d holds, or -1;
 *     local_counts [R][G + B]: rows of each local expert (home experts, then
 *       the slots) -- the local cu_seqlens is their exclusive scan;
 *     remote_reads [R]: rows of remote experts left without a slot (weights
 *       read from the home rank).
 *   Every destination gets exactly S*K rows.  The plan depends on the counts
 *   only (deterministic), so every rank computes the same plan from gathered
 *   counts.  No device work; returns MOE_OK or an argument error.
 */
MOE_API int moe_ep_plan(int R, int E, int S, int K, int B, const int32_t* counts, int32_t* piece_count,
                        int32_t* piece_offset, int32_t* slot_expert, int32_t* local_counts,
                        int32_t* remote_reads);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
