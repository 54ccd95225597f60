/*
 * deltanet.h -- C ABI of the MI355X (gfx950) DeltaNet delta-rule library.
 *
 * The operation.  Per (batch b, head h) the state S is a d_k x d_v matrix and
 * every token t, in order, does
 *     v_old = k_t S                    (read what the state holds at key k_t)
 *     u_t   = beta_t (v_t - v_old)     (gated delta)
 *     S     = S + k_t^T u_t            (outer-product write)
 *     o_t   = q_t S                    (read after the write, no scale)
 * This is the sequential delta-rule prefill loop of the page
 * "GPT-2 から Kimi K3 まで、AI モデルの進化を解説" (news.ainew.jp), section
 * "DeltaNet (Parallelizing linear transformers with delta rule)", and, at
 * one token, that page's layer forward in "DeltaNet (Fast weight
 * programmers)".  The chunked forward computes exactly this result (up to
 * floating-point rounding) with the chunkwise-parallel generalised-Householder
 * form the same section describes.
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    never frees or retains them.  Tensors are dense, row-major, C-contiguous,
 *    with the shapes given below (last index fastest), 16-byte aligned.
 *  - beta and the state are always fp32.  q, k, v are fp32 or bf16
 *    (in_dtype).  o is fp32 or bf16 (out_dtype).
 *  - Work is enqueued on `stream` (0 = the null stream) and the call returns
 *    without synchronising.  Faults during execution surface at the caller's
 *    next synchronisation.
 *  - Every argument is validated before anything is launched: on any non-OK
 *    status nothing has been launched and no output has been written.
 *  - The library keeps no state between calls besides loaded code objects;
 *    calls on different streams with disjoint buffers may run concurrently.
 */
#ifndef DELTANET_H_
#define DELTANET_H_

#include <stddef.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DN_OK = 0,
  DN_ERR_NULL_ARG = 1,     /* a required pointer is NULL                       */
  DN_ERR_BAD_SHAPE = 2,    /* a size is negative/zero where it must be >= 1     */
  DN_ERR_UNSUPPORTED = 3,  /* d_k, d_v, C or a dtype outside the built set      */
  DN_ERR_MISALIGNED = 4,   /* a pointer is not 16-byte aligned                  */
  DN_ERR_ALIASING = 5,     /* an output overlaps an input it must not overlap   */
  DN_ERR_WORKSPACE = 6,    /* workspace given but smaller than required         */
  DN_ERR_HIP = 7           /* a HIP runtime call failed; see deltanet_last_hip_error */
} dn_status;

/* Element types of q, k, v (in_dtype) and o (out_dtype).  The last
 * enumerator only gives the type the range of an int, so that a value
 * outside the set reaches the argument checks (DN_ERR_UNSUPPORTED). */
typedef enum { DN_F32 = 0, DN_BF16 = 1, DN_DTYPE_RANGE_ = 0x7fffffff } dn_dtype;

/*
 * Chunkwise-parallel delta-rule forward over a whole sequence.
 *
 *   q, k   : [B, H, L, d_k]   in_dtype
 *   v      : [B, H, L, d_v]   in_dtype
 *   beta   : [B, H, L]        fp32, per-token write strength
 *   S0     : [B, H, d_k, d_v] fp32 initial state, or NULL for the zero state
 *   o      : [B, H, L, d_v]   out_dtype, written (o_t read after token t's write).
 *            The kernels compute o in fp32; out_dtype = DN_BF16 stores it
 *            rounded to nearest even, which alone moves an element by up to
 *            2^-9 |o| (measured against the exact result: 1.2e-2 RMS(o) at
 *            B=4 H=12 L=2048 d=64, 2.5e-2 at B=2 H=16 L=8192 d=128 with beta
 *            = 1 heads, 1.7e-2 at B=1 H=32 L=65536 d=128, the largest errors
 *            being the roundings of the largest outputs).  Where an error
 *            bound of 2e-2 RMS(o) has to hold at such sizes, take DN_F32.
 *   S_final: [B, H, d_k, d_v] fp32 state after the last token, or NULL to skip.
 *            S_final may be the same buffer as S0 (in-place state update);
 *            any other overlap with an input is rejected.
 *   L      : any length >= 0 (L = 0 copies S0 (or zeros) to S_final; a
 *            ragged last chunk is handled by masking, an exact no-op).
 *   d_k, d_v in {64, 128}; C (chunk length) in {64, 128}.
 *   workspace: device scratch of at least deltanet_chunk_fwd_workspace_bytes()
 *            bytes, or NULL to let the library allocate and free it on
 *            `stream` (stream-ordered).  Its contents on entry do not matter.
 *
 * Returns DN_OK or the first failing check's status.
 */
int deltanet_chunk_fwd(const void* q, const void* k, const void* v, const float* beta,
                       const float* S0, void* o, float* S_final,
                       int B, int H, int L, int d_k, int d_v, int C,
                       dn_dtype in_dtype, dn_dtype out_dtype,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace deltanet_chunk_fwd needs for these sizes (0 if the
 * sizes are invalid or unsupported). */
size_t deltanet_chunk_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int C,
                                          dn_dtype in_dtype);

/*
 * deltanet_chunk_fwd that allocates nothing, for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc.  Same arguments, layouts and result as
 * deltanet_chunk_fwd, without the workspace arguments: the scratch comes from
 * a fixed area of DN_NOALLOC_SCRATCH_BYTES compiled into the library, one per
 * GPU, held from the library's load until the process ends.  No call makes
 * hipMalloc, hipFree or any other allocation.
 *
 *  - Sizes whose workspace (deltanet_chunk_fwd_workspace_bytes) exceeds
 *    DN_NOALLOC_SCRATCH_BYTES return DN_ERR_WORKSPACE and launch nothing
 *    (64 MiB holds e.g. B*H = 32 heads of L = 8192 at C = 64 with bf16
 *    inputs, not the L = 65536, 32-head long-context shape).
 *  - The area is found on the device `stream` belongs to; its address is
 *    looked up (hipGetSymbolAddress) on the first call for each device, so
 *    make one call per device before capturing a graph.
 *  - All calls on one GPU share its area and it keeps the previous call's
 *    contents (nothing in it has to start cleared).  Calls that overlap in
 *    time on one GPU (other streams, other threads) race on it: serialise them.
 */
#define DN_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int deltanet_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const float* beta,
                               const float* S0, void* o, float* S_final,
                               int B, int H, int L, int d_k, int d_v, int C,
                               dn_dtype in_dtype, dn_dtype out_dtype, hipStream_t stream);

/*
 * One decode step for B sequences x H heads (the recurrence at one token),
 * updating the state in place.
 *
 *   q, k : [B, H, d_k] in_dtype;  v : [B, H, d_v] in_dtype
 *   beta : [B, H] fp32
 *   S    : [B, H, d_k, d_v] fp32, read and overwritten with the new state
 *   o    : [B, H, d_v] out_dtype, o = q S_new
 *   d_k, d_v in {64, 128}.  o must not overlap S or any input.
 */
int deltanet_decode_step(const void* q, const void* k, const void* v, const float* beta,
                         float* S, void* o, int B, int H, int d_k, int d_v,
                         dn_dtype in_dtype, dn_dtype out_dtype, hipStream_t stream);

/*
 * Gated forms (Gated DeltaNet).  The article "How a Baseten Engineer Traced 7
 * Years of Attention Mechanism Evolution" (wpnews.pro / dev.to), section on
 * Gated DeltaNet, adds a decay alpha in [0, 1] that is applied to the old
 * state first, after which the precise delta write acts on the decayed
 * state; alpha = 1 is the plain delta rule, alpha = 0 wipes the memory.  Per
 * (b, h) and token t, in order:
 *     S     = alpha_t S
 *     v_old = k_t S
 *     u_t   = beta_t (v_t - v_old)
 *     S     = S + k_t^T u_t
 *     o_t   = q_t S
 * Arguments are those of the plain entry points plus alpha, fp32, one value
 * per token: [B, H, L] for the chunked forward, [B, H] for the decode step.
 * alpha must be 16-byte aligned and may not overlap an output; values outside
 * [0, 1] are not checked (the product is then not a decay).  A zero alpha is
 * taken as a factor of about 1e-38 inside a chunk (the kernels sum
 * log(alpha), floored at log(FLT_MIN)), which is a wipe to within fp32.
 * The chunked forward's workspace is larger than the plain one's: query it
 * with deltanet_gated_chunk_fwd_workspace_bytes().  With L = 0, alpha may be
 * NULL.  Status codes and every other rule are as for the plain calls.
 */
int deltanet_gated_chunk_fwd(const void* q, const void* k, const void* v, const float* alpha,
                             const float* beta, const float* S0, void* o, float* S_final,
                             int B, int H, int L, int d_k, int d_v, int C,
                             dn_dtype in_dtype, dn_dtype out_dtype,
                             void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace deltanet_gated_chunk_fwd needs (0 if the sizes are
 * invalid or unsupported). */
size_t deltanet_gated_chunk_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int C,
                                                dn_dtype in_dtype);

/* One gated decode step, S updated in place; o = q S_new.  alpha: [B, H] fp32. */
int deltanet_gated_decode_step(const void* q, const void* k, const void* v, const float* alpha,
                               const float* beta, float* S, void* o, int B, int H,
                               int d_k, int d_v, dn_dtype in_dtype, dn_dtype out_dtype,
                               hipStream_t stream);

/*
 * Gradient of the chunked forward (training).  The pages present the chunked
 * form as the way to train the delta rule in linear time but print no
 * backward pass; this one is the reverse-mode derivative of the forward
 * above (plain delta rule, no gate).  Given the gradients of a loss with
 * respect to the forward's outputs, it returns those with respect to its
 * inputs:
 *   q, k   : [B, H, L, d_k]  in_dtype;   v : [B, H, L, d_v] in_dtype
 *   beta   : [B, H, L] fp32;  S0 : [B, H, d_k, d_v] fp32 or NULL (zero state)
 *   dO     : [B, H, L, d_v] fp32, dL/do
 *   dS_final: [B, H, d_k, d_v] fp32, dL/dS_final, or NULL (zero)
 *   dq, dk : [B, H, L, d_k] fp32;  dv : [B, H, L, d_v] fp32;
 *   dbeta  : [B, H, L] fp32;       dS0 : [B, H, d_k, d_v] fp32 or NULL (not
 *            written)
 * The forward is recomputed inside (nothing from a previous forward call is
 * needed).  64-token chunks whatever C names (C must still be 64 or 128);
 * with bf16 inputs the recomputed forward runs on the chunked forward's
 * kernels at 128-token chunks.  bf16 inputs run every product on bf16 matrix
 * cores with each fp32 operand split into a (hi, lo) bf16 pair; fp32 inputs
 * run fp32 vector-ALU kernels.  Outputs may not overlap inputs or one
 * another.  The workspace holds, per 64-token chunk, the entering state and
 * the exit gradient (2 d_k d_v floats) besides per-chunk matrices, and the
 * forward's T per 128-token chunk: query deltanet_chunk_bwd_workspace_bytes().
 */
int deltanet_chunk_bwd(const void* q, const void* k, const void* v, const float* beta,
                       const float* S0, const float* dO, const float* dS_final,
                       float* dq, float* dk, float* dv, float* dbeta, float* dS0,
                       int B, int H, int L, int d_k, int d_v, int C, dn_dtype in_dtype,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace deltanet_chunk_bwd needs (0 if the sizes are invalid or
 * unsupported). */
size_t deltanet_chunk_bwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int C,
                                          dn_dtype in_dtype);

/*
 * Per-dimension decay (KDA).  The same article describes Kimi Linear's KDA as
 * Gated DeltaNet with the scalar gate turned into a vector: each dimension of
 * the memory forgets at its own rate.  The gate acts on the key dimension,
 * the rows of S.  Per (b, h) and token t, in order:
 *     S     = diag(alpha_t) S          alpha_t in [0, 1]^{d_k}
 *     v_old = k_t S
 *     u_t   = beta_t (v_t - v_old)
 *     S     = S + k_t^T u_t
 *     o_t   = q_t S
 * Arguments are those of the gated entry points with alpha one fp32 per key
 * dimension: [B, H, L, d_k] for the chunked forward, [B, H, d_k] for the
 * decode step.  alpha must be 16-byte aligned and may not overlap an output;
 * zeros are floored inside a chunk as for the scalar gate.  The chunked
 * forward runs in 64-token chunks whatever C names (the result does not
 * depend on the chunk size; C must still be 64 or 128): for bf16 inputs its
 * scan and most of its prep on bf16 matrix cores with split operands, for
 * fp32 inputs on fp32 vector-ALU kernels.  Its workspace is larger than the other forms':
 * query deltanet_kda_chunk_fwd_workspace_bytes().  With L = 0, alpha may be
 * NULL.
 */
int deltanet_kda_chunk_fwd(const void* q, const void* k, const void* v, const float* alpha,
                           const float* beta, const float* S0, void* o, float* S_final,
                           int B, int H, int L, int d_k, int d_v, int C,
                           dn_dtype in_dtype, dn_dtype out_dtype,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace deltanet_kda_chunk_fwd needs (0 if the sizes are invalid
 * or unsupported). */
size_t deltanet_kda_chunk_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int C,
                                              dn_dtype in_dtype);

/* One decode step with per-dimension decay, S updated in place; o = q S_new.
 * alpha: [B, H, d_k] fp32. */
int deltanet_kda_decode_step(const void* q, const void* k, const void* v, const float* alpha,
                             const float* beta, float* S, void* o, int B, int H,
                             int d_k, int d_v, dn_dtype in_dtype, dn_dtype out_dtype,
                             hipStream_t stream);

/*
 * The layer's feature maps (page "GPT-2 から Kimi K3 まで、AI モデルの進化を解説",
 * section "DeltaNet (Fast weight programmers)": before the delta rule the
 * layer maps its projections to
 *     q = normalise(silu(q_raw)),  k = normalise(silu(k_raw)),
 *     beta = sigmoid(beta_logit),
 * with silu(x) = x sigmoid(x) and normalise(x) = x / max(||x||_2, 1e-12)
 * along d_k, as PyTorch's F.normalize).  The maps are evaluated in fp32; q
 * and k are stored in `dtype` (bf16: rounded to nearest, ties to even),
 * beta in fp32.  Elements of a row beyond ~1e19 overflow its fp32 sum of
 * squares (the row then maps to zeros).
 *
 *   q_raw, k_raw, q_hat, k_hat : [B, H, L, d_k] dtype
 *   beta_logit, beta            : [B, H, L] fp32
 *   d_k in {64, 128}.  Every pointer is required when B H L > 0.  An output
 *   may be the very buffer of its own input (in place); any other overlap is
 *   rejected.
 */
int deltanet_feature_prep(const void* q_raw, const void* k_raw, const float* beta_logit,
                          void* q_hat, void* k_hat, float* beta,
                          int B, int H, int L, int d_k, dn_dtype dtype, hipStream_t stream);

/*
 * The chunked forward fed by the raw projections: the feature maps above,
 * then the plain (alpha == NULL) or gated (alpha given) chunked forward on the
 * mapped q, k, beta.  Arguments are those of deltanet_chunk_fwd /
 * deltanet_gated_chunk_fwd with q_raw, k_raw in place of q, k and
 * beta_logit in place of beta.  The mapped operands live in the workspace,
 * which is therefore larger: query it with
 * deltanet_chunk_fwd_features_workspace_bytes(..., gated = alpha != NULL).
 */
int deltanet_chunk_fwd_features(const void* q_raw, const void* k_raw, const void* v,
                                const float* alpha, const float* beta_logit, const float* S0,
                                void* o, float* S_final,
                                int B, int H, int L, int d_k, int d_v, int C,
                                dn_dtype in_dtype, dn_dtype out_dtype,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace deltanet_chunk_fwd_features needs (gated != 0 when
 * alpha will be given; 0 if the sizes are invalid or unsupported). */
size_t deltanet_chunk_fwd_features_workspace_bytes(int B, int H, int L, int d_k, int d_v, int C,
                                                   dn_dtype in_dtype, int gated);

/*
 * One decode step fed by the raw projections: the feature maps are applied
 * inside the step's kernel (no extra memory traffic), then the plain
 * (alpha == NULL) or gated step.  Arguments are those of
 * deltanet_decode_step / deltanet_gated_decode_step with q_raw, k_raw and
 * beta_logit in place of q, k and beta.
 */
int deltanet_decode_step_features(const void* q_raw, const void* k_raw, const void* v,
                                  const float* alpha, const float* beta_logit, float* S, void* o,
                                  int B, int H, int d_k, int d_v, dn_dtype in_dtype, dn_dtype out_dtype,
                                  hipStream_t stream);

/*
 * The gated linear recurrence: the additive write with a decay, per (b, h)
 * and token t, in order,
 *     S   = e^{g_t} S + k_t^T v_t
 *     o_t = q_t S                      (read after the write, no scale)
 * It is the printed chunked linear-attention form of the page above, section
 * "DeltaNet (Parallelizing linear transformers with delta rule)", with the
 * decay of the Gated DeltaNet article on the state: the delta rule without
 * its read before the write.
 *
 *   q, k     : [B, H_qk, L, d_k] in_dtype.  State head h reads q and k of head
 *              h / (H / H_qk); H must be a multiple of H_qk (H_qk = H: every
 *              head its own).
 *   v        : [B, H, L, d_v] in_dtype
 *   log_decay: [B, H, L] fp32, the decay's natural logarithm, or NULL (no
 *              decay).  0 keeps the state, -inf wipes it: a log decay of -inf
 *              at its first token separates a document from the one before it
 *              in the same row.  At a call's first token it drops S0 whatever
 *              that holds, infinities or memory never written too.  Values
 *              above 0 are not checked (the product is then no decay).
 *   S0       : [B, H, d_k, d_v] fp32 or NULL (zero state)
 *   o        : [B, H, L, d_v] out_dtype, written
 *   S_final  : [B, H, d_k, d_v] fp32 or NULL; may be the buffer of S0.
 *   L >= 0 (L = 0 copies S0, or zeros, to S_final).  d_k, d_v in {64, 128}.
 * The result does not depend on how the sequence is cut into chunks, so
 * there is no chunk argument.  bf16 inputs run on the bf16 matrix cores, every
 * fp32 operand as a sum of bf16 pieces: three, which are all of its 24 bits, on
 * the way to fp32 results (S_final always is one), two, which leave 2^-17 of a
 * term, for what only reaches a bf16 o.  fp32 inputs run on the fp32 ones.  A
 * non-finite q, k or v row makes outputs of its 64-token chunk (tokens 64 n to
 * 64 n + 63, earlier ones too) and, from k or v, the states after it
 * non-finite (a wipe behind it in the same call does not clear them): padding
 * has to be finite.  workspace, workspace_bytes, stream,
 * status codes and every other rule: as for deltanet_chunk_fwd; the workspace
 * holds one fp32 state per segment that the sequence is cut into, and may be
 * 0 bytes.
 */
int deltanet_linear_chunk_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                              const float* S0, void* o, float* S_final,
                              int B, int H, int H_qk, int L, int d_k, int d_v,
                              dn_dtype in_dtype, dn_dtype out_dtype,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace deltanet_linear_chunk_fwd needs (0 also if the sizes are
 * invalid or unsupported). */
size_t deltanet_linear_chunk_fwd_workspace_bytes(int B, int H, int H_qk, int L, int d_k, int d_v,
                                                 dn_dtype in_dtype);

/*
 * Its gradient, from the gradients of o and S_final:
 *   dO        : [B, H, L, d_v] in_dtype;  dS_final: [B, H, d_k, d_v] fp32 or NULL (zero)
 *   dq, dk    : [B, H_qk, L, d_k] in_dtype (heads that share q and k are added in fp32)
 *   dv        : [B, H, L, d_v] in_dtype
 *   dlog_decay: [B, H, L] fp32, the gradient of log_decay (exactly 0 where
 *               log_decay is -inf), or NULL (not written; required to be NULL
 *               when log_decay is).  Summed over the pairs (write before t, read
 *               at t or after) alone, so documents that a wipe separates do not
 *               reach each other's.  What a 64-token chunk passes through is a
 *               difference of sums, off by about 2^-24 of the largest
 *               <state, its gradient> of the document: not small against a single
 *               token's gradient whose decay leaves less than that of the state
 *               (where a chunk leaves below 2^-64 there is no such term).
 *   dS0       : [B, H, d_k, d_v] fp32 or NULL (not written)
 * Nothing from a forward call is needed.  Outputs may not overlap inputs or
 * one another.
 */
int deltanet_linear_chunk_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                              const float* S0, const void* dO, const float* dS_final,
                              void* dq, void* dk, void* dv, float* dlog_decay, float* dS0,
                              int B, int H, int H_qk, int L, int d_k, int d_v, dn_dtype in_dtype,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace deltanet_linear_chunk_bwd needs (0 if the sizes are
 * invalid or unsupported). */
size_t deltanet_linear_chunk_bwd_workspace_bytes(int B, int H, int H_qk, int L, int d_k, int d_v,
                                                 dn_dtype in_dtype);

/* One token of the gated linear recurrence, S updated in place; o = q S_new.
 * q, k: [B, H_qk, d_k], v, o: [B, H, d_v], log_decay: [B, H] fp32 or NULL;
 * B H up to 2^24 - 1. */
int deltanet_linear_decode_step(const void* q, const void* k, const void* v, const float* log_decay,
                                float* S, void* o, int B, int H, int H_qk, int d_k, int d_v,
                                dn_dtype in_dtype, dn_dtype out_dtype, hipStream_t stream);

/*
 * Per-head norm of q and k and rotation by position, in one pass (the map in
 * front of a core that deltanet_feature_prep's silu and L2 norm are for the
 * delta rule).  For each row x of d_k elements:
 *     n = x / sqrt(mean(x^2) + eps) o weight         (norm = 0: n = x o weight)
 *     pair j of n's first d_rot elements is turned by p inv_freq[j] radians:
 *       (a, b) -> (a cos - b sin, a sin + b cos)
 * Pair j is elements (j, j + d_rot / 2), or (2 j, 2 j + 1) when interleaved;
 * elements from d_rot on are not turned.  p is the token's position on pair
 * j's axis: axis a owns sections[a] pairs, in order (one axis: all of them).
 *
 *   q_raw, k_raw  : rows (b, h, l) of [B, H_q, L, d_k] and [B, H_k, L, d_k], dtype, at
 *                   strides[0] b + strides[1] h + strides[2] l elements (strides NULL:
 *                   dense).  So q and k can be read out of a fused projection's rows.
 *                   Strides are >= 0 and keep every row 16-byte aligned; 0 repeats a row.
 *                   H_k may be 0 (q only).
 *   q_weight, k_weight: [d_k] fp32 or NULL (ones)
 *   positions     : [n_axes, B, L] int32;  inv_freq: [d_rot / 2] fp32;
 *   sections      : HOST array of n_axes counts adding up to d_rot / 2 (NULL for one axis)
 *                   Both device pointers may be NULL when d_rot = 0 (no rotation).
 *   q_hat, k_hat  : [B, H_q, L, d_k], [B, H_k, L, d_k] dtype, dense, written
 *   d_k in {64, 128}; d_rot a multiple of 8, 0 .. d_k; n_axes 1 .. 4; eps >= 0.
 * Evaluated in fp32, angles in fp64 (any int32 position).  Rows beyond ~1e19
 * overflow their fp32 sum of squares (the row then maps to zeros); with eps = 0,
 * rows below ~1e-18 lose bits of it, and rows of zeros or below ~1e-23 are not
 * finite.  Sizes beyond
 * one launch are DN_ERR_UNSUPPORTED: with H_q + H_k <= 4, 2^24 - 1 times 32 tokens
 * of 64 elements or 16 of 128, with more heads that many fewer.
 */
int deltanet_qk_norm_rope(const void* q_raw, const long long* q_strides,
                          const void* k_raw, const long long* k_strides,
                          const float* q_weight, const float* k_weight,
                          const int* positions, const float* inv_freq,
                          const int* sections, int n_axes, void* q_hat, void* k_hat,
                          int B, int H_q, int H_k, int L, int d_k, int d_rot,
                          int norm, int interleaved, float eps, dn_dtype dtype, hipStream_t stream);

/*
 * Its gradient, from dq_hat, dk_hat ([B, H, L, d_k] dtype, dense):
 *   dq_raw, dk_raw: rows at strides of their own (NULL: dense), written; their rows may
 *                   not share elements, and may be the q and k parts of one buffer of
 *                   token rows (equal batch and token strides, q and k apart in the row)
 *   dq_weight, dk_weight: [d_k] fp32 or NULL (not written), summed over all rows
 *                   in an order that does not change from call to call
 * The rest as above.
 */
int deltanet_qk_norm_rope_bwd(const void* q_raw, const long long* q_strides,
                              const void* k_raw, const long long* k_strides,
                              const float* q_weight, const float* k_weight,
                              const int* positions, const float* inv_freq,
                              const int* sections, int n_axes,
                              const void* dq_hat, const void* dk_hat,
                              void* dq_raw, const long long* dq_strides,
                              void* dk_raw, const long long* dk_strides,
                              float* dq_weight, float* dk_weight,
                              int B, int H_q, int H_k, int L, int d_k, int d_rot,
                              int norm, int interleaved, float eps, dn_dtype dtype,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace deltanet_qk_norm_rope_bwd needs (0 also if the sizes are
 * invalid or unsupported). */
size_t deltanet_qk_norm_rope_bwd_workspace_bytes(int B, int H_q, int H_k, int L, int d_k,
                                                 dn_dtype dtype);

/*
 * Short causal convolution: each channel's last K tokens, in front of a layer's
 * recurrence.  With x_e the K - 1 rows kept from before a sequence followed by its rows,
 *     p_t = bias + sum_j weight[:, j] o x_e[t + j],  j = 0 .. K - 1
 *     y_t = silu(p_t)   (silu = 0: p_t)
 * and the rows kept behind the sequence are x_e's last K - 1 (so a sequence may be
 * taken in pieces, and by single tokens).
 *
 *   x      : rows of [B, L, D] dtype at x_strides[0] b + x_strides[1] t elements
 *            (x_strides: HOST array of 2, or NULL: dense), e.g. a part of a fused
 *            projection's rows.  Strides are >= 0 and keep rows 16-byte aligned.
 *   weight : [D, K] fp32;  bias: [D] fp32 or NULL
 *   state0 : [n, K - 1, D] dtype, the kept rows in front, oldest first, or NULL (zeros)
 *   cu_seqlens: NULL: B sequences of L tokens (n = B, n_seq is not used).  Or [n_seq + 1]
 *            int32 on the device, B = 1: sequence i holds rows cu_seqlens[i] to
 *            cu_seqlens[i + 1] - 1 (none if they are equal), n = n_seq.  They may not
 *            fall and lie in 0 .. L; where they do not, the results are not defined,
 *            but nothing outside the tensors is read or written.
 *   y      : [B, L, D] dtype, dense, written.  Rows that no sequence holds (in front of
 *            the first, behind the last) become zeros, so that a product over all
 *            rows stays finite.
 *   state  : [n, K - 1, D] dtype, the kept rows behind, or NULL (not written); not state0
 *   D a multiple of 8; K in {2, 3, 4}.  Evaluated in fp32.
 */
int deltanet_short_conv_fwd(const void* x, const long long* x_strides, const float* weight, const float* bias,
                            const void* state0, const int* cu_seqlens, void* y, void* state,
                            int B, int L, int D, int K, int n_seq, int silu, dn_dtype dtype, hipStream_t stream);

/*
 * Its gradient, from dy ([B, L, D] dtype, dense) and dstate ([n, K - 1, D] dtype or NULL):
 *   dx     : [B, L, D] dtype, dense (zeros in rows that no sequence holds)
 *   dweight: [D, K] fp32;  dbias: [D] fp32 or NULL (not written); both summed in an order
 *            that does not change from call to call
 *   dstate0: [n, K - 1, D] dtype or NULL (not written)
 */
int deltanet_short_conv_bwd(const void* x, const long long* x_strides, const float* weight, const float* bias,
                            const void* state0, const int* cu_seqlens, const void* dy, const void* dstate,
                            void* dx, float* dweight, float* dbias, void* dstate0,
                            int B, int L, int D, int K, int n_seq, int silu, dn_dtype dtype,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);
/* Bytes of workspace deltanet_short_conv_bwd needs (0 also if the sizes are invalid or unsupported). */
size_t deltanet_short_conv_bwd_workspace_bytes(int B, int L, int D, int K);

/* One token of every sequence: x [B, D] (rows at *x_stride elements, NULL: dense), y [B, D];
 * state [B, K - 1, D] is moved on by a row in place. */
int deltanet_short_conv_step(const void* x, const long long* x_stride, const float* weight, const float* bias,
                             void* state, void* y, int B, int D, int K, int silu, dn_dtype dtype, hipStream_t stream);

/*
 * Selective state space scan: a recurrence with a decay of its own for every channel d
 * and state n, set by the token.  Per sequence, token t in order:
 *     dt_t = softplus(raw_t + dt_bias)           (softplus = 0: raw_t + dt_bias)
 *     h[d, n] = exp(dt_t[d] A[d, n]) h[d, n] + dt_t[d] u_t[d] B_t[n]
 *     y_t[d]  = (sum_n C_t[n] h[d, n] + D_skip[d] u_t[d]) silu(z_t[d])     (without z: no last factor)
 *
 *   u, dt, z: rows of [B, L, D] dtype; dt is raw; z may be NULL.  B, C (Bm, Cm): rows of
 *            [B, L, N] dtype, shared by all channels.  strides: HOST array of 10, (batch, token)
 *            of u, dt, Bm, Cm, z in this order, or NULL (all dense); rules as above.
 *   A      : [D, N] fp32, negative (with a positive one no state may grow by more than 2^127 over
 *            a call);  D_skip, dt_bias: [D] fp32 or NULL (zeros)
 *   h0     : [n, D, N] fp32 or NULL (zeros);  cu_seqlens, n_seq, n: as above
 *   y      : [B, L, D] dtype, dense, written (zeros in rows that no sequence holds)
 *   hT     : [n, D, N] fp32, the states behind, or NULL; may be h0 (in place)
 *   D a multiple of 8; N in {8, 16, 32}.  Evaluated in fp32; L = 0 copies h0.
 * A state that is not finite, and tokens that are not, stay in their own channel and sequence.
 * A long sequence of few channels is cut into segments whose states are joined: the decay over
 * a segment is then exp(A sum dt), and a state that overflows inside the sequence need not do
 * so at the same token as in a walk from its start.
 */
int deltanet_selective_scan_fwd(const void* u, const void* dt, const void* Bm, const void* Cm, const void* z,
                                const long long* strides, const float* A, const float* D_skip, const float* dt_bias,
                                const float* h0, const int* cu_seqlens, void* y, float* hT,
                                int B, int L, int D, int N, int n_seq, int softplus, dn_dtype dtype,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);
/* Bytes of workspace deltanet_selective_scan_fwd needs (packed: whether cu_seqlens is given; 0
 * also if the sizes are invalid or unsupported). */
size_t deltanet_selective_scan_fwd_workspace_bytes(int B, int L, int D, int N, int packed, int n_seq);

/*
 * Its gradient, from dy ([B, L, D] dtype, dense) and dhT ([n, D, N] fp32 or NULL):
 *   du, ddt (of raw), dz: [B, L, D] dtype, dense; dB, dC: [B, L, N] dtype, dense (zeros in rows that
 *            no sequence holds); dz is not used without z
 *   dA     : [D, N] fp32;  dD_skip, ddt_bias: [D] fp32 or NULL (not written);  dh0: [n, D, N] fp32 or NULL
 * Nothing from a forward call is needed.  All sums run in an order that does not change from
 * call to call.  D (N + 2) is at most 2^28 - 16.  The workspace holds two states ([D, N] fp32) for
 * every 16 tokens or part of them in a segment, and dB's and dC's parts, [B, L, N] fp32 each for
 * every 64 channels.
 */
int deltanet_selective_scan_bwd(const void* u, const void* dt, const void* Bm, const void* Cm, const void* z,
                                const long long* strides, const float* A, const float* D_skip, const float* dt_bias,
                                const float* h0, const int* cu_seqlens, const void* dy, const float* dhT,
                                void* du, void* ddt, void* dB, void* dC, void* dz,
                                float* dA, float* dD_skip, float* ddt_bias, float* dh0,
                                int B, int L, int D, int N, int n_seq, int softplus, dn_dtype dtype,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);
size_t deltanet_selective_scan_bwd_workspace_bytes(int B, int L, int D, int N, int packed, int n_seq);

/* One token of every sequence: u, dt, z, y [B, D], Bm, Cm [B, N] (strides: HOST array of 5 row strides
 * in the same order, or NULL); h [B, D, N] fp32 updated in place. */
int deltanet_selective_scan_step(const void* u, const void* dt, const void* Bm, const void* Cm, const void* z,
                                 const long long* strides, const float* A, const float* D_skip, const float* dt_bias,
                                 float* h, void* y, int B, int D, int N, int softplus, dn_dtype dtype, hipStream_t stream);

/*
 * Root-mean-square norm of rows with the residual's addition, in front of a layer's projections:
 *     total = x + residual, rounded to residual_dtype;   y = total / sqrt(mean(total^2) + eps) o weight
 *   x      : [rows, D] dtype;  residual, total: [rows, D] residual_dtype, both NULL for the norm of x
 *            alone.  total may be residual, or x where the types agree (in place).
 *   weight : [D] fp32 or NULL (ones)
 *   y      : [rows, D] dtype;  or, with scale ([rows] fp32), 8-bit e4m3 values with
 *            y = value * scale: scale is the row's largest magnitude / 448 (1 for a row of zeros)
 *   D a multiple of 8, up to 32768; dtype = DN_F32 needs residual_dtype = DN_F32.  Evaluated in fp32:
 * rows beyond ~1e19 overflow their sum of squares (y is then zeros); with eps = 0 rows below ~1e-19
 * lose digits of theirs, and a row of zeros is not finite.  What is not finite stays in its row.
 */
int deltanet_add_rms_norm(const void* x, const void* residual, const float* weight, void* total, void* y, float* scale,
                          int rows, int D, float eps, dn_dtype dtype, dn_dtype residual_dtype, hipStream_t stream);

/*
 * Its gradient, from dy ([rows, D] dtype) and dtotal ([rows, D] residual_dtype, what reaches total from
 * elsewhere, or NULL); total as the forward wrote it (the norm of x alone: x, with residual_dtype = dtype):
 *   dx     : [rows, D] dtype;  dresidual: the same in residual_dtype, or NULL (not written)
 *   dweight: [D] fp32 or NULL (not written), summed in an order that does not change from call to call
 * The workspace is used for dweight alone.
 */
int deltanet_add_rms_norm_bwd(const void* total, const float* weight, const void* dy, const void* dtotal,
                              void* dx, void* dresidual, float* dweight, int rows, int D, float eps,
                              dn_dtype dtype, dn_dtype residual_dtype,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);
size_t deltanet_add_rms_norm_bwd_workspace_bytes(int rows, int D);

/* Static, NUL-terminated description of a status code. */
const char* deltanet_status_string(int status);

/* The hipError_t behind the last DN_ERR_HIP returned on this thread (0 if none). */
int deltanet_last_hip_error(void);

/*
 * Profiling hook.  Between deltanet_profile_start() and
 * deltanet_profile_stop() on the same host thread, every kernel the library
 * launches from that thread is bracketed by two HIP events recorded on the
 * call's stream.  deltanet_profile_stop() waits for those events and writes,
 * per kernel slot, the summed elapsed milliseconds and the launch count
 * (nslots entries each; slots: 0 = chunk WY-prep kernel, 1 = chunk scan
 * kernel, 2 = decode kernel, 3 = feature-map kernel; the backward's kernels:
 * 4 = prep, 5 = forward state pass (for bf16 inputs the chunked forward's
 * prep and scan kernels at 128-token chunks, counted together), 6 = reverse
 * state pass, 7 = per-chunk matrix gradients, 8 = dq / dk; for bf16 inputs one
 * kernel computes both the matrix gradients and dq / dk and is counted in
 * slot 8; the gated linear recurrence's: 9 = segment sums and their
 * combination, 10 = outputs, 11 = the backward's walks and decay gradient,
 * 12 = decode; the q / k norm with rotation: 13 = forward, 14 = backward; the
 * short convolution: 15 = forward and step, 16 = backward; the selective scan:
 * 17 = forward, 18 = backward, 19 = step; the norm with addition: 20, 21).
 * Recording adds two event records per launch.
 * deltanet_profile_start() creates the thread's events up front (4096,
 * enough for 2048 launches; more are created as needed), so it can take a
 * few milliseconds the first time; it returns DN_ERR_HIP if that fails.
 */
int deltanet_profile_start(void);
int deltanet_profile_stop(double* ms_per_slot, int* launches_per_slot, int nslots);

/* Library version as major*10000 + minor*100 + patch. */
int deltanet_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DELTANET_H_ */
