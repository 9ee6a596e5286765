/*
 * moe.h — C ABI of the routed mixture-of-experts expert computation on
 * AMD Instinct MI355X (gfx950).
 *
 * The operation (kernelindex.com operation pages):
 *   "Sparse expert dispatch and combine" (description): tokens routed to an
 *     expert are extracted, pass through a gate_up projection, a gated GLU
 *     with clamping and a down projection, and are accumulated back into the
 *     output rows of their tokens.
 *   "MoE training token repeat and expert computation" (description): every
 *     token is repeated once per chosen expert, each expert selects its rows,
 *     runs a SwiGLU FFN, and the routing weights scale the expert outputs
 *     before the sum over the chosen experts.
 *   "MoE expert parallel execution backward" (description): gradients with
 *     respect to hidden_states, topk_weights and the gate, up and down weights.
 *
 * Notation: T tokens, H hidden size, I intermediate size, E experts, K experts
 * per token (the workload lines' hidden_size, intermediate_size,
 * num_local_experts / num_experts / n_routed_experts, num_experts_per_tok).
 * S = T*K slots; slot s = t*K + k is the k-th copy of token t.
 *
 *   out[t] = sum_k w[t,k] * Wd[e] . phi(Wgu[e] . x_t),   e = ids[t,k]
 *
 * phi splits the 2I gate_up outputs into gate g and up u (layout flag) and is
 *   MOE_SWIGLU:      g * sigmoid(g) * u
 *   MOE_CLAMPED_GLU: gc = min(g, L), uc = clamp(u, -L, L),
 *                    (uc + 1) * gc * sigmoid(alpha * gc)     (L = clamp_limit)
 *                    (min and clamp of a NaN are NaN)
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers, row-major, contiguous, 16-byte
 *     aligned.  hidden/out/d_out/d_hidden [T,H]; w_gate_up/d_w_gate_up
 *     [E,2I,H]; w_gate/w_up/d_w_gate/d_w_up [E,I,H]; w_down/d_w_down
 *     [E,H,I]; topk_ids int32 [T,K]; topk_weights/d_topk_weights fp32 [T,K];
 *     router logits/d_logits fp32 [T,E].  Activations, weights and
 *     d_hidden have the descriptor's dtype (bf16 or fp32); the weight
 *     gradients have its grad_dtype.
 *   - The caller owns every buffer.  The library never allocates device
 *     memory, never frees, and keeps no pointer after a call returns.
 *   - Outputs are fully overwritten (never accumulated).
 *   - Calls are asynchronous on `stream` and never synchronise the host,
 *     except moe_check_device_status.  Calls are re-entrant given distinct
 *     workspaces; two calls sharing one workspace must be stream-ordered.
 *   - Host-checkable errors are reported before any launch, with nothing
 *     written: MOE_ERR_INVALID_ARG (null pointer where one is required,
 *     T<0, K<1, E<1, H<1, I<1, bad enum, misaligned pointer),
 *     MOE_ERR_UNSUPPORTED (H or I not a multiple of 8, E > 1024, K > 64,
 *     S >= 2^31), MOE_ERR_WORKSPACE (ws_bytes below the required size).
 *     A failed kernel launch returns MOE_ERR_HIP.
 *   - An expert id outside [0,E) is found on the device and its slot is
 *     dropped: out, d_hidden and the weight gradients are those of the same
 *     call with that slot's routing weight set to zero, its d_topk_weights
 *     entry is 0, and routing places it after every valid slot (inv_pos -1).
 *     A count is kept in the workspace and moe_check_device_status reports
 *     MOE_ERR_BAD_EXPERT_ID.  No memory outside the caller's buffers is
 *     touched for such an id.
 *   - T = 0 is valid: nothing is launched for the activations; the forward
 *     and backward entry points and moe_router clear the workspace status
 *     word (so moe_check_device_status reports MOE_OK for the call), and the
 *     backward entry points write zero weight gradients.
 *   - Entry points that take router logits or separate gate/up tensors
 *     (moe_router, moe_fwd_logits, moe_router_bwd, moe_fwd_sep, moe_bwd_sep)
 *     follow the same conventions; their own comments give the shapes.
 */
#ifndef MOE_MI355X_H
#define MOE_MI355X_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,
  MOE_ERR_UNSUPPORTED = 2,
  MOE_ERR_WORKSPACE = 3,
  MOE_ERR_HIP = 4,
  MOE_ERR_BAD_EXPERT_ID = 5
} moe_status_t;

typedef enum { MOE_BF16 = 0, MOE_F32 = 1 } moe_dtype_t;
typedef enum { MOE_SWIGLU = 0, MOE_CLAMPED_GLU = 1 } moe_act_t;
/* CONCAT: rows [0,I) of w_gate_up[e] are the gate, rows [I,2I) the up
 * projection.  INTERLEAVED: row 2j is gate column j, row 2j+1 up column j. */
typedef enum { MOE_GU_CONCAT = 0, MOE_GU_INTERLEAVED = 1 } moe_gu_layout_t;

typedef struct {
  int64_t T, H, I, E, K;
  int32_t dtype;      /* moe_dtype_t */
  int32_t act;        /* moe_act_t */
  int32_t gu_layout;  /* moe_gu_layout_t */
  float clamp_limit;  /* L of the clamped GLU (7.0 for the gpt-oss shapes) */
  float glu_alpha;    /* alpha of the clamped GLU (1.702) */
  int32_t grad_dtype; /* moe_dtype_t of d_w_gate_up / d_w_down (accumulation is
                         always fp32; MOE_F32 stores the fp32 sums) */
} moe_desc_t;

/* Sizes in bytes of the workspaces moe_fwd and moe_bwd need, and of the
 * optional `saved` buffer (the gate_up projection outputs Z, fp32 [S,2I] in
 * expert-sorted slot order) that moe_fwd can fill for moe_bwd.  Any output
 * pointer may be NULL.
 * The routing part of both workspaces is moe_route_workspace_size(). */
moe_status_t moe_workspace_size(const moe_desc_t* desc, size_t* fwd_ws,
                                size_t* bwd_ws, size_t* saved_bytes);
moe_status_t moe_route_workspace_size(const moe_desc_t* desc, size_t* route_ws);

/* Expert histogram and stable grouping of the slots by expert — the "masked
 * indexing" / "sparse token extraction" step of the pages' descriptions.
 * Outputs (device, int32):
 *   counts[E]       slots routed to each expert
 *   offsets[E+1]    exclusive prefix sum of counts
 *   sorted_slot[S]  slots in expert order; ascending slot id inside an expert;
 *                   slots with an id outside [0,E) last, in ascending order
 *   inv_pos[S]      position of slot s in sorted_slot (-1 for a bad id)
 * Bit-exact and deterministic.  Any of the four outputs may be NULL (then not
 * written).  ws: at least moe_route_workspace_size() bytes. */
moe_status_t moe_route(const moe_desc_t* desc, const int32_t* topk_ids,
                       int32_t* counts, int32_t* offsets, int32_t* sorted_slot,
                       int32_t* inv_pos, void* ws, size_t ws_bytes,
                       hipStream_t stream);

/* Router + routing in one pipeline.  The pages take the top-k expert ids and
 * weights as inputs of the layer ("MoE expert parallel execution backward"
 * lists topk_weights among the tensors it differentiates); this produces
 * them from router logits the way the workloads define routing: the softmax
 * over a token's E logits, its K largest entries, renormalised to sum to one
 * (equal, up to rounding, to the softmax of the K largest logits).
 *   logits        fp32 [T,E] (read only; finite values expected: an infinite
 *                 logit can give NaN weights, and a token whose remaining
 *                 logits are all NaN gets id -1 in the slots left, reported
 *                 as MOE_ERR_BAD_EXPERT_ID by moe_check_device_status)
 *   topk_ids      int32 [T,K] out: ids by descending logit; equal logits in
 *                 ascending id (bit-exact: ids are decided by comparisons of
 *                 the fp32 logits only)
 *   topk_weights  fp32 [T,K] out: exp(l_k - l_0) / sum_j exp(l_j - l_0) in
 *                 fp32, summed in k order (a few ulp from the exact value)
 *   counts, offsets, sorted_slot, inv_pos: as moe_route for these ids (each
 *                 may be NULL).
 * Requires K <= E (else MOE_ERR_INVALID_ARG).  ws: at least
 * moe_route_workspace_size() bytes; the routing it leaves there is the one
 * moe_fwd would compute from topk_ids. */
moe_status_t moe_router(const moe_desc_t* desc, const float* logits,
                        int32_t* topk_ids, float* topk_weights, int32_t* counts,
                        int32_t* offsets, int32_t* sorted_slot, int32_t* inv_pos,
                        void* ws, size_t ws_bytes, hipStream_t stream);

/* Forward: out [T,H] = sum_k w[t,k] * FFN_{ids[t,k]}(hidden[t]).
 * Routing, gate_up projection with the gated activation, down projection with
 * the routing weight, and a deterministic per-token sum over the K slots
 * (fp32, k order, one rounding).  `saved` may be NULL; if given, it receives
 * Z for moe_bwd and `saved_bytes` (its size) must be at least the
 * saved_bytes of moe_workspace_size, else MOE_ERR_WORKSPACE (nothing
 * launched). */
moe_status_t moe_fwd(const moe_desc_t* desc, const void* hidden,
                     const int32_t* topk_ids, const float* topk_weights,
                     const void* w_gate_up, const void* w_down, void* out,
                     void* saved, size_t saved_bytes, void* ws,
                     size_t ws_bytes, hipStream_t stream);

/* Backward of moe_fwd given d_out = dL/dout [T,H]:
 *   d_hidden [T,H], d_topk_weights fp32 [T,K] (<d_out[t], expert output of
 *   slot s>), d_w_gate_up [E,2I,H] (gate rows = dW_gate, up rows = dW_up, in
 *   w_gate_up's layout), d_w_down [E,H,I].  Weight gradients are accumulated
 *   in fp32 over the tokens and stored in grad_dtype; an expert with no slots
 *   gets exact zeros.  `saved` is the buffer moe_fwd filled for the same
 *   inputs, or NULL (then Z is recomputed); when given, `saved_bytes` (its
 *   size) must be at least moe_workspace_size's saved_bytes, else
 *   MOE_ERR_WORKSPACE (nothing launched). */
moe_status_t moe_bwd(const moe_desc_t* desc, const void* hidden,
                     const int32_t* topk_ids, const float* topk_weights,
                     const void* w_gate_up, const void* w_down,
                     const void* d_out, const void* saved, size_t saved_bytes,
                     void* d_hidden, float* d_topk_weights, void* d_w_gate_up,
                     void* d_w_down, void* ws, size_t ws_bytes,
                     hipStream_t stream);

/* Forward from router logits [T,E] (fp32): moe_router's top-k and weights
 * (written to topk_ids [T,K] and topk_weights [T,K] for the backward), then
 * moe_fwd on them in the same call.  Same outputs, workspace, `saved` /
 * `saved_bytes` and errors as moe_fwd (plus K <= E). */
moe_status_t moe_fwd_logits(const moe_desc_t* desc, const void* hidden,
                            const float* logits, const void* w_gate_up,
                            const void* w_down, void* out, int32_t* topk_ids,
                            float* topk_weights, void* saved,
                            size_t saved_bytes, void* ws, size_t ws_bytes,
                            hipStream_t stream);

/* Gradient of the router's weights with respect to its logits, given
 * d_topk_weights fp32 [T,K] (from moe_bwd): d_logits fp32 [T,E] with
 *   d_logits[t, ids[t,k]] = w[t,k] * (g[t,k] - sum_j w[t,j] g[t,j])
 * and zero for experts not chosen (the choice is piecewise constant in the
 * logits).  Ids outside [0,E) contribute nothing; a repeated id of one token
 * receives the sum of its terms.  fp32, one writer per element. */
moe_status_t moe_router_bwd(const moe_desc_t* desc, const int32_t* topk_ids,
                            const float* topk_weights,
                            const float* d_topk_weights, float* d_logits,
                            hipStream_t stream);

/* Separate gate and up weights ("MoE expert parallel execution backward",
 * description, differentiates gate, up and down weights as three tensors):
 * w_gate, w_up [E,I,H] in place of w_gate_up, and in moe_bwd_sep d_w_gate,
 * d_w_up [E,I,H] (grad_dtype) in place of d_w_gate_up; gate and up rows are
 * then g = w_gate[e].x and u = w_up[e].x, and desc->gu_layout is ignored.
 * Everything else (outputs, workspace sizes, `saved`, errors) is as for
 * moe_fwd / moe_bwd; a `saved` buffer filled by moe_fwd_sep is meant for
 * moe_bwd_sep (its Z columns are the I gate columns, then the I up columns).
 * w_up and d_w_up must not be NULL. */
moe_status_t moe_fwd_sep(const moe_desc_t* desc, const void* hidden,
                         const int32_t* topk_ids, const float* topk_weights,
                         const void* w_gate, const void* w_up,
                         const void* w_down, void* out, void* saved,
                         size_t saved_bytes, void* ws, size_t ws_bytes,
                         hipStream_t stream);
moe_status_t moe_bwd_sep(const moe_desc_t* desc, const void* hidden,
                         const int32_t* topk_ids, const float* topk_weights,
                         const void* w_gate, const void* w_up,
                         const void* w_down, const void* d_out,
                         const void* saved, size_t saved_bytes,
                         void* d_hidden, float* d_topk_weights, void* d_w_gate,
                         void* d_w_up, void* d_w_down, void* ws,
                         size_t ws_bytes, hipStream_t stream);

/* Forward for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  Same
 * computation, outputs, `saved` / `saved_bytes` and errors as moe_fwd, with
 * the workspace taken from an array of MOE_NOALLOC_SCRATCH_BYTES that the
 * library holds on each GPU it runs on (part of its code object, kept until
 * the process ends); the call allocates nothing.
 *   - Shapes whose moe_fwd workspace (moe_workspace_size's fwd_ws) exceeds
 *     MOE_NOALLOC_SCRATCH_BYTES return MOE_ERR_WORKSPACE before any device
 *     call (for H = I = 2880, E = 128, K = 4: up to about 3800 slots).
 *   - Every call on one GPU uses that GPU's one array: calls that overlap on
 *     a GPU (other streams, other threads) race and must be ordered by the
 *     caller.  Nothing in the array needs to start at zero.
 *   - bad_ids (device int32, nullable) receives the number of slots with an
 *     id outside [0,E) (the status moe_check_device_status reports for
 *     moe_fwd's workspace). */
#define MOE_NOALLOC_SCRATCH_BYTES (64u << 20)
moe_status_t moe_fwd_noalloc(const moe_desc_t* desc, const void* hidden,
                             const int32_t* topk_ids,
                             const float* topk_weights, const void* w_gate_up,
                             const void* w_down, void* out, void* saved,
                             size_t saved_bytes, int32_t* bad_ids,
                             hipStream_t stream);

/* Forward for a few tokens (decoding): T <= MOE_FEW_MAX_TOKENS, else
 * MOE_ERR_UNSUPPORTED.  Computes moe_fwd's out without its routing pass and
 * without `saved` (no backward), by kernels sized for one or two slots an
 * expert: an active expert's weights are read once for each 64 of its slots.
 * a = phi(..) is rounded to the activations' type as in moe_fwd; sums over H,
 * I and K are fp32 in a fixed order (not moe_fwd's order, so the two agree to
 * rounding, not bit for bit).  A bf16 call with more than 4 slots an expert
 * (T K > 4 E) and T K H I above 2e9 runs moe_fwd's kernels, with their order
 * and workspace.
 * MOE_ERR_UNSUPPORTED also where 64 rows of the weights, hidden, or a [S,I]
 * reach 2^31 bytes.  ws: at least moe_few_workspace_size() bytes (its first
 * word is the status that moe_check_device_status reports); nothing in it has
 * to start at zero.  Bad expert ids, T = 0, streams and errors as for
 * moe_fwd.  moe_fwd_few_logits takes router logits [T,E] and writes the ids
 * and weights it chose, as moe_fwd_logits does. */
#define MOE_FEW_MAX_TOKENS 128
moe_status_t moe_few_workspace_size(const moe_desc_t* desc, size_t* ws_bytes);
moe_status_t moe_fwd_few(const moe_desc_t* desc, const void* hidden,
                         const int32_t* topk_ids, const float* topk_weights,
                         const void* w_gate_up, const void* w_down, void* out,
                         void* ws, size_t ws_bytes, hipStream_t stream);
moe_status_t moe_fwd_few_logits(const moe_desc_t* desc, const void* hidden,
                                const float* logits, const void* w_gate_up,
                                const void* w_down, void* out,
                                int32_t* topk_ids, float* topk_weights,
                                void* ws, size_t ws_bytes, hipStream_t stream);

/* Weight rows in 4-bit microscaled floating point (the OCP MXFP4 element and
 * scale formats): blocks of 32 consecutive columns share one E8M0 scale byte
 * s, each element is an E2M1 code c (sign, 2 exponent bits, 1 mantissa bit:
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) and stands for
 * c * 2^(s - 127); s = 255 makes its block NaN.
 *   codes  uint8 [rows, cols/2]: column 2i in the low, 2i+1 in the high half
 *   scales uint8 [rows, cols/32]
 * moe_mx_quantize: s - 127 = max(floor(log2(max |w|)) - 2, -127) over the
 * block, the code is the nearest to w / 2^(s-127), ties to the even code,
 * magnitudes beyond 6 become 6; a block with an infinity or NaN gets s = 255
 * and zero codes.  moe_mx_dequantize gives the values the codes stand for:
 * exact in bf16 and fp32, except that a value of 2^128 and more (scale byte
 * 253 with |c| of 4 and 6, 254 with 2 and more; moe_mx_quantize writes neither
 * byte) is infinite in both.  w: [rows, cols] of `dtype` (moe_dtype_t); cols a
 * multiple of 32, else MOE_ERR_UNSUPPORTED; rows = 0 does nothing. */
moe_status_t moe_mx_quantize(const void* w, int32_t dtype, int64_t rows,
                             int64_t cols, void* codes, void* scales,
                             hipStream_t stream);
moe_status_t moe_mx_dequantize(const void* codes, const void* scales,
                               int32_t dtype, int64_t rows, int64_t cols,
                               void* w, hipStream_t stream);

/* Forward on expert weights in that form: gu_codes [E,2I,H/2], gu_scales
 * [E,2I,H/32] in the descriptor's gate/up layout, d_codes [E,H,I/2], d_scales
 * [E,H,I/32]; hidden, out and a = phi(..) are bf16 and products accumulate in
 * fp32.  Computes what moe_fwd computes on the weights moe_mx_dequantize
 * gives.  dtype must be MOE_BF16, H and I multiples of 32 and at most 14336,
 * and hidden below 2^31 bytes, else MOE_ERR_UNSUPPORTED.  ws: at least
 * moe_mx_workspace_size() bytes.
 * Up to MOE_FEW_MAX_TOKENS tokens run as in moe_fwd_few, an expert's weights
 * read once for each 32 of its slots.  Grouped products over routed slots run
 * more tokens, and of those calls the ones with T K > 4 E and T K H I above
 * 2e9, with T K > 64 E, with H or I above 8192, or with T K + max(H, I) above
 * 15872.  The two sum in different orders and need different workspaces.
 * Everything else as for moe_fwd (no `saved`, no backward);
 * moe_mx_fwd_logits is to it as moe_fwd_logits to moe_fwd. */
moe_status_t moe_mx_workspace_size(const moe_desc_t* desc, size_t* ws_bytes);
moe_status_t moe_mx_fwd(const moe_desc_t* desc, const void* hidden,
                        const int32_t* topk_ids, const float* topk_weights,
                        const void* gu_codes, const void* gu_scales,
                        const void* d_codes, const void* d_scales, void* out,
                        void* ws, size_t ws_bytes, hipStream_t stream);
moe_status_t moe_mx_fwd_logits(const moe_desc_t* desc, const void* hidden,
                               const float* logits, const void* gu_codes,
                               const void* gu_scales, const void* d_codes,
                               const void* d_scales, void* out,
                               int32_t* topk_ids, float* topk_weights,
                               void* ws, size_t ws_bytes, hipStream_t stream);

/* ---- The operators around the routed experts.  Same conventions as above:
 * device pointers, row-major, contiguous, 16-byte aligned, every buffer the
 * caller's, asynchronous on `stream`, nothing launched after an error. */

/* Gated feed-forward block that every token passes: the shared expert beside
 * the routed ones, or a dense layer.
 *   out[t] = add[t] + s_t * Wd . phi(Wgu . x_t),   s_t = sigmoid(gate[t])
 * with the descriptor's phi, gate/up layout and types; its E and K must be 1
 * (else MOE_ERR_INVALID_ARG).  x, out, add [T,H]; w_gate_up [2I,H]; w_down
 * [H,I]; gate fp32 [T].  add may be NULL (zero) and may be out; gate may be
 * NULL (s = 1).
 *   - H and I at most 2^20, H I at most 2^28, T at most 2^30 and at most 2^23
 *     tiles of 256 x 256 in [T, max(2I, H)], else MOE_ERR_UNSUPPORTED.
 *   - a = phi(..) is rounded to the activations' type as the second product's
 *     operand; sums are fp32; out is rounded once.
 *   - Up to 16 tokens (bf16) or 512 (fp32) without `saved` run on kernels that
 *     read the weights once and make no tiles; their order of sums is their
 *     own.
 *   - `saved` (nullable) receives the gate and up values (fp32, in an order of
 *     the library's) for moe_ffn_bwd; saved_bytes below the required size:
 *     MOE_ERR_WORKSPACE.
 * moe_ffn_bwd, given d_out [T,H]: d_x [T,H], d_gate fp32 [T] (with gate;
 * s (1 - s) <d_out, y>), d_w_gate_up [2I,H], d_w_down [H,I] in grad_dtype
 * (fp32 sums over the tokens); the gradient of add is d_out.  `saved`: what
 * moe_ffn_fwd left for the same inputs, or NULL (recomputed).  T = 0 writes
 * zero weight gradients.  In fp32 the products of more than 512 tokens, and
 * the backward pass, are those of moe_fwd / moe_bwd with one expert.
 * Any output of moe_ffn_workspace_size may be NULL. */
moe_status_t moe_ffn_workspace_size(const moe_desc_t* desc, size_t* fwd_ws,
                                    size_t* bwd_ws, size_t* saved_bytes);
moe_status_t moe_ffn_fwd(const moe_desc_t* desc, const void* x,
                         const void* w_gate_up, const void* w_down,
                         const float* gate, const void* add, void* out,
                         void* saved, size_t saved_bytes, void* ws,
                         size_t ws_bytes, hipStream_t stream);
moe_status_t moe_ffn_bwd(const moe_desc_t* desc, const void* x,
                         const void* w_gate_up, const void* w_down,
                         const float* gate, const void* d_out,
                         const void* saved, size_t saved_bytes, void* d_x,
                         float* d_gate, void* d_w_gate_up, void* d_w_down,
                         void* ws, size_t ws_bytes, hipStream_t stream);

/* Norms around a block, rms(v)^2 = mean(v^2) + eps over a row, all in fp32
 * from the stored values, rounded once.
 *   moe_norm_fwd:      y = w * x / rms(x)
 *   moe_norm_bwd:      d_x = d_add + its gradient for d_y;  d_w fp32 [H]
 *   moe_residual_fwd:  n = w_post * h / rms(h)  (n = h if w_post is NULL)
 *                      x_new = x + scale * gate * n
 *                      y = w_next * x_new / rms(x_new), from x_new before it
 *                      is rounded  (w_next NULL: y is not written)
 *   moe_residual_bwd:  given d_x_new and d_y, and x_new as it was stored,
 *                      t = d_x_new + the norm's gradient for d_y;
 *                      d_x = t, d_h, d_gate, d_w_post, d_w_next of the above
 * x, h, x_new, y and their gradients [T,H] and the weights [H] have the
 * descriptor's dtype; d_w, d_w_post, d_w_next are fp32 [H].
 * gate, of that dtype, is [T] (MOE_GATE_ROW: one value for a row), [H]
 * (MOE_GATE_COLUMN) or [T,H] (MOE_GATE_FULL); d_gate has its shape, fp32 for
 * the two that are sums, the descriptor's dtype for MOE_GATE_FULL.
 * NULL is allowed for d_add and d_x_new (zero), w_post and w_next (no such
 * norm; its gradient's pointer is then ignored, as d_y is without w_next), and
 * gate with MOE_GATE_NONE.  x_new may be x, and d_x may be d_add or d_x_new.
 * H a multiple of 8, at most 16384, and T at most 2^30, else
 * MOE_ERR_UNSUPPORTED.  With an eps of 0 a row of zeros has no rms and is NaN.
 * T = 0 writes zeros to the weights' (and a column gate's) gradients.
 * ws (backward): moe_norm_workspace_size() bytes.  Deterministic. */
typedef enum {
  MOE_GATE_NONE = 0,
  MOE_GATE_ROW = 1,
  MOE_GATE_COLUMN = 2,
  MOE_GATE_FULL = 3
} moe_gate_t;
typedef struct {
  int64_t T, H;
  int32_t dtype;     /* moe_dtype_t */
  int32_t gate_kind; /* moe_gate_t; MOE_GATE_NONE for moe_norm_* */
  float scale;       /* of the residual step */
  float eps;         /* >= 0 */
} moe_norm_desc_t;
moe_status_t moe_norm_workspace_size(const moe_norm_desc_t* desc,
                                     size_t* bwd_ws);
moe_status_t moe_norm_fwd(const moe_norm_desc_t* desc, const void* x,
                          const void* w, void* y, hipStream_t stream);
moe_status_t moe_norm_bwd(const moe_norm_desc_t* desc, const void* x,
                          const void* w, const void* d_y, const void* d_add,
                          void* d_x, float* d_w, void* ws, size_t ws_bytes,
                          hipStream_t stream);
moe_status_t moe_residual_fwd(const moe_norm_desc_t* desc, const void* x,
                              const void* h, const void* w_post,
                              const void* gate, const void* w_next,
                              void* x_new, void* y, hipStream_t stream);
moe_status_t moe_residual_bwd(const moe_norm_desc_t* desc, const void* x_new,
                              const void* h, const void* w_post,
                              const void* gate, const void* w_next,
                              const void* d_x_new, const void* d_y, void* d_x,
                              void* d_h, void* d_gate, float* d_w_post,
                              float* d_w_next, void* ws, size_t ws_bytes,
                              hipStream_t stream);

/* Newton-Schulz orthogonalisation of E stacked M x N updates (moe_bwd's
 * weight gradients are such stacks):
 *   X = G / (|G| + eps), then `steps` times
 *   X <- a X + b (X X^T) X + c (X X^T)^2 X
 * with |G| the 2-norm of a matrix's elements, which drives the singular values
 * towards one.  moe_orthogonalize writes X to out (out_dtype).  moe_muon_step
 * takes a gradient G, a momentum fp32 and weights (w_dtype), [E,M,N] each:
 *   m_out = momentum m + G,  U = G + momentum m_out (nesterov) or m_out
 *   w_out = (1 - decay) w - lr X(U)
 * m_out may be m and w_out may be w.
 * Iterates are held in 22 bits, of which the products take 11 (fp16), with
 * fp32 sums: after five steps of the usual coefficients X is about 1e-3 from the
 * exact iteration in the 2-norm, whatever the update's rank, before it is
 * rounded to its type (up to 4e-3 where a few roundings are all of it: a side
 * below 64, an update with elements in a few rows or columns only); the norm is
 * summed in 64 bits.  Coefficients must keep the iterates' singular values,
 * which start at most 1, at most 3 and b x + c x^2 and a + b x + c x^2 at most
 * 14.6 in size over their squares (checked; the usual 3.4445, -4.775, 2.0315
 * reach 1.21, 2.81 and 3.45), else MOE_ERR_UNSUPPORTED.  A NaN or infinity
 * makes its matrix's X NaN; a zero matrix stays zero, with an eps of 0 too.
 * M and N multiples of 8, at most 2^20, E at most 65535, at most 2^23 tiles of
 * 256 x 256 (128 x 128 where a side is below 64) in all the matrices, 1 to 64
 * steps, else MOE_ERR_UNSUPPORTED (negative E, M or N, M or N of 0, eps or dtypes
 * that do not exist: MOE_ERR_INVALID_ARG).  E = 0 does nothing. */
typedef struct {
  int64_t E, M, N;
  int32_t dtype;     /* of G: moe_dtype_t */
  int32_t out_dtype; /* of out, or of w and w_out */
  int32_t steps;
  float a, b, c;
  float eps;         /* >= 0 */
} moe_ortho_desc_t;
typedef struct {
  float lr, momentum, decay;
  int32_t nesterov; /* 0 or 1 */
} moe_muon_t;
moe_status_t moe_ortho_workspace_size(const moe_ortho_desc_t* desc,
                                      size_t* ws_bytes);
moe_status_t moe_orthogonalize(const moe_ortho_desc_t* desc, const void* g,
                               void* out, void* ws, size_t ws_bytes,
                               hipStream_t stream);
moe_status_t moe_muon_step(const moe_ortho_desc_t* desc,
                           const moe_muon_t* opt, const void* w,
                           const void* g, const float* m, void* w_out,
                           float* m_out, void* ws, size_t ws_bytes,
                           hipStream_t stream);

/* Synchronises `stream` and reports MOE_ERR_BAD_EXPERT_ID if the last
 * routing done in `ws` met an id outside [0,E), else MOE_OK. */
moe_status_t moe_check_device_status(const void* ws, hipStream_t stream);

/* Static, human-readable name of a status code. */
const char* moe_status_str(moe_status_t status);

/* Kernel timing (instrumentation for benchmarks).  While enabled, every
 * kernel the library launches is bracketed by two HIP events recorded on the
 * launch stream (events come from a library-owned pool of `max_launches`
 * pairs, created on enable; later launches are not timed).  moe_timing_read
 * synchronises those events and returns, per kernel name, the number of
 * timed launches and their summed duration; it resets the pool.
 * Not thread-safe; meant for one benchmarking thread. */
typedef struct {
  char name[48];
  int32_t launches;
  double total_ms;
} moe_kernel_time_t;
moe_status_t moe_timing_enable(int32_t max_launches);
moe_status_t moe_timing_disable(void);
moe_status_t moe_timing_read(moe_kernel_time_t* out, int32_t max_entries,
                             int32_t* n_entries);

#ifdef __cplusplus
}
#endif
#endif /* MOE_MI355X_H */
