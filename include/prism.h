/*
 * prism.h -- C ABI of the PRISM layer hot path on AMD MI355X (gfx950).
 *
 * The layer is the one described by the web summary "Technical Summary: PRISM
 * (Parallel Residual Iterative Sequence Model)" (gist.science, paper
 * 2602.10796), sections cited as §n below:
 *
 *   Stage 1 (§2.2): u_t = sum_{j=0..3} conv[h, :, j] * v_{t-j}      (ShortConv anchor)
 *   Stage 2 (§2.2): r^(1) = v_t - u_t; for l = 1..L:
 *                   k^(l) = W_k^(l) u_t, p^(l) = W_p^(l) u_t,
 *                   beta^(l) = sigmoid(w_beta^(l) . u_t),
 *                   delta^(l) = GELU(p^(l) * r^(l)), r^(l+1) = r^(l) - delta^(l)
 *   Write   (§2.2): B_t = beta_t v_t k_t^T + sum_l beta^(l) delta^(l) k^(l)^T
 *   Forget  (§2.1): A_t = alpha_t (I - beta_t k_t k_t^T)   (Gated-DeltaNet form)
 *   Update  (§2.1): S_t = S_{t-1} A_t + B_t
 *   Readout        : o_t = S_t q_t
 * With L = 0 the layer is Gated DeltaNet (§3, item 3).  GELU is the exact erf
 * form.  The base term beta_t v_t k_t^T of the write, r^(1) = v - u, the conv
 * over v of width 4 (tap j multiplies v_{t-j}), the gate beta^(l) as a
 * sigmoid of w_beta^(l) . u and the readout are readings of passages the
 * summary leaves open; the library implements exactly the formulas above.
 *
 * Conventions common to every entry point
 * ---------------------------------------
 * - All tensor pointers are DEVICE pointers, contiguous, row-major, 16-byte
 *   aligned (the later sections name what they take beside that).  The caller
 *   owns every buffer, including the workspace.  The library allocates no
 *   device memory and keeps no pointer after a call.
 * - Work is enqueued asynchronously on `stream`; nothing synchronises the
 *   host.  Buffers must stay alive until the stream has finished the work.
 * - Every argument is validated on the host before any HIP call; a failed
 *   check returns a non-zero status and enqueues nothing.
 *   prism_last_error() then returns a message naming the argument.
 * - NaN / Inf inputs are not checked; they propagate.
 * - Results are deterministic: the same inputs and descriptor give bitwise
 *   identical outputs (all reductions in a fixed order; atomics only where
 *   the gated recurrence's tiles take their places and pass their states on,
 *   which changes no order of operations).
 * - Functions are thread-safe except while kernel timing is enabled
 *   (prism_timing_begin .. prism_timing_end).
 */
#ifndef PRISM_H_
#define PRISM_H_

#include <stddef.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PRISM_OK = 0,
  PRISM_ERR_NULL = 1,        /* a required pointer is NULL                      */
  PRISM_ERR_SHAPE = 2,       /* a size is out of range (B, T, H < 1, ...)       */
  PRISM_ERR_UNSUPPORTED = 3, /* valid but outside the compiled envelope         */
  PRISM_ERR_ALIGN = 4,       /* a pointer is not 16-byte aligned                */
  PRISM_ERR_WORKSPACE = 5,   /* workspace NULL or smaller than required         */
  PRISM_ERR_HIP = 6          /* a HIP launch failed; see prism_last_error()     */
} prism_status;

typedef enum {
  PRISM_F32 = 0,  /* q, k, v, o, weights, taps, dO, dq, dk, dv in float32  */
  PRISM_BF16 = 1  /* the same tensors in bfloat16 (round-to-nearest-even)  */
} prism_dtype;

/* Refinement step activation (summary §2.2 "Residual Update"): the step
 * correction is delta = GELU(p * r) (the method) or delta = p * r (the
 * ablation without the nonlinearity). */
typedef enum {
  PRISM_ACT_GELU = 0,
  PRISM_ACT_IDENTITY = 1,
  PRISM_ACT_SILU = 2       /* z sigmoid(z), of prism_short_conv alone */
} prism_activation;

/* Problem descriptor.
 *   B, T, H    batch, sequence length, heads            (each >= 1;
 *              H * dk <= 4194304)
 *   dk, dv     key / value head dimension; must be equal, in {16, 32, 64, 128}
 *              for PRISM_BF16 and {16, 32, 64} for PRISM_F32
 *   L          refinement steps, 0 <= L <= 8
 *   chunk      tokens per chunk of the parallel scan, in {16, 32, 64}
 *              (PRISM_F32 also needs dk * chunk <= 2048); any T >= 1 is
 *              accepted (the last chunk may be partial)
 *   conv_width ShortConv width; must be 4
 *   dtype      storage type of the dtype-typed tensors (see prism_dtype)
 *   activation refinement step activation, PRISM_ACT_GELU (0, the method's
 *              step) or PRISM_ACT_IDENTITY
 *   conv_offset ShortConv tap offset: 0 = tap j multiplies v_{t-j} (the
 *              current token and the three before it), 1 = tap j multiplies
 *              v_{t-1-j} (strictly past tokens, the ones the state S_{t-1}
 *              has seen; summary §2.2 Stage 1)
 *   packed_tokens  with cu_seqlens (packed batch, below): N, the number of
 *              token rows in the packed tensors; must be >= 0.  Ignored for
 *              a dense batch.
 * A zero-initialised tail (activation = conv_offset = 0) is the method as
 * described.  activation and conv_offset are ignored when L = 0.           */
typedef struct {
  int B, T, H, dk, dv, L, chunk, conv_width;
  prism_dtype dtype;
  int activation, conv_offset;
  int packed_tokens;
} prism_desc;

/* Tensor layouts (element type "dt" = desc->dtype; f32 = float32):
 *   q, k        [B, T, H, dk]  dt      v, o, dO   [B, T, H, dv]  dt
 *   alpha, beta [B, T, H]      f32     alpha in (0, 1], beta in [0, 1]
 *   Wk          [H, L, dk, dv] dt      k^(l) = Wk[h, l] u   (row i . u)
 *   Wp          [H, L, dv, dv] dt      p^(l) = Wp[h, l] u
 *   wbeta       [H, L, dv]     dt      beta^(l) = sigmoid(wbeta[h, l] . u)
 *   conv        [H, dv, 4]     dt      tap j multiplies v_{t-j} (j = 0: current token),
 *                                      or v_{t-1-j} with conv_offset = 1
 *   conv_hist   [B, 4, H, dv]  dt      v_{-4} .. v_{-1}: the four values before the
 *                                      sequence, oldest first (v's own layout)
 *   S0, ST      [B, H, dv, dk] f32     state entering / leaving the sequence
 *   dST, dS0    [B, H, dv, dk] f32
 *   dq, dk, dv  as q, k, v     dt
 *   dalpha, dbeta [B, T, H]    f32
 *   dWk, dWp, dwbeta, dconv    f32, layouts of Wk, Wp, wbeta, conv
 *   dconv_hist  [B, 4, H, dv]  f32
 * q and k are used as given (callers normalise them if they wish).  With
 * L = 0, Wk, Wp, wbeta, conv (and their gradients) may be NULL.
 *
 * Packed batches (variable lengths).  With cu_seqlens (a device array of
 * B + 1 int32 offsets, 4-byte aligned; NULL = dense) the token tensors q, k,
 * v, o, dO, dq, dk, dv are [N, H, d] and alpha, beta, dalpha, dbeta [N, H],
 * N = desc->packed_tokens, sequence b being tokens cu_seqlens[b] ..
 * cu_seqlens[b+1] - 1; desc->T is then the longest length (it sizes the
 * workspaces).  Meant: cu_seqlens[0] = 0, non-decreasing, cu_seqlens[B] = N,
 * every length <= desc->T (lengths of 0 are allowed: S_T = S0).  The offsets
 * are read on the device only: before any kernel uses them, a sanitising
 * pass replaces them by c'_i = max_{j <= i} min(max(cu_seqlens[j], 0), N),
 * and sequences longer than T are cut at T.  Offsets outside the contract
 * therefore give results for those clamped sequences (rows of o and of the
 * gradients outside every clamped sequence are not written), but no access
 * outside the N rows.  conv_hist, S0, ST and their gradients stay per
 * sequence.  A packed batch computes exactly what each sequence would
 * compute alone.
 *
 * Continuation.  A sequence split over several calls gives the same result
 * as one call when each call after the first receives S0 = the previous ST
 * and conv_hist = the previous call's conv_hist_out (summary §2.1: the state
 * carries the past; §2.2 Stage 1: the ShortConv reads the last few values).
 * NULL conv_hist means zeros before the sequence. */

/* Workspace sizes in bytes for a descriptor; *bytes = 0 on error.  The
 * training pair (below) keeps most intermediates in its saved buffer, so its
 * entry points need the (smaller) sizes of the *_train_workspace queries. */
prism_status prism_forward_workspace(const prism_desc* desc, size_t* bytes);
prism_status prism_backward_workspace(const prism_desc* desc, size_t* bytes);
prism_status prism_forward_train_workspace(const prism_desc* desc, size_t* bytes);
prism_status prism_backward_train_workspace(const prism_desc* desc, size_t* bytes);

/* Forward pass: o = readout of S_1..S_T, ST = S_T (ST may be NULL).
 * S0 may be NULL (zero initial state); conv_hist may be NULL (zeros).
 * conv_hist_out (may be NULL) receives the four values of v before the end
 * of the sequence (from conv_hist, or zeros, where T < 4); it may be the same
 * buffer as conv_hist, which is then updated in place after every read. */
prism_status prism_forward(const prism_desc* desc, const void* q, const void* k, const void* v,
                           const float* alpha, const float* beta, const void* Wk, const void* Wp,
                           const void* wbeta, const void* conv, const float* S0,
                           const void* conv_hist, const int* cu_seqlens, void* o, float* ST,
                           void* conv_hist_out, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/* Backward pass: gradients of <dO, o> + <dST, S_T> with respect to every
 * input.  Stateless: recomputes what it needs from the forward inputs.
 * dST may be NULL (zero).  dS0 and dconv_hist may be NULL; each is written
 * when given (dconv_hist is the gradient with respect to conv_hist, zero
 * when L = 0).  Every other gradient pointer is required (weight / tap
 * gradients only when L > 0).  Gradients are written, not accumulated. */
prism_status prism_backward(const prism_desc* desc, const void* q, const void* k, const void* v,
                            const float* alpha, const float* beta, const void* Wk, const void* Wp,
                            const void* wbeta, const void* conv, const float* S0,
                            const void* conv_hist, const int* cu_seqlens, const void* dO,
                            const float* dST, void* dq, void* dk, void* dv, float* dalpha,
                            float* dbeta, float* dWk, float* dWp, float* dwbeta, float* dconv,
                            float* dS0, float* dconv_hist, void* workspace,
                            size_t workspace_bytes, hipStream_t stream);

/* Training pair (saved intermediates).  prism_forward_train computes what
 * prism_forward computes and also keeps, in the caller-owned `saved` buffer,
 * the intermediates the backward needs: the refinement pairs (k^(l), w^(l))
 * of every token, and per chunk the affine map M^T, the decay sum g_C, the
 * chunk-entry state S_c, the readout operand Qt and the solve results U^T,
 * W_k^T (summary §2.1-2.2 as rewritten per chunk).  prism_backward_train then
 * returns the same gradients as prism_backward with the same inputs, starting
 * from those intermediates instead of recomputing the forward.
 *   saved:     device buffer of prism_saved_bytes() bytes, 256-byte aligned,
 *              written by prism_forward_train, read by prism_backward_train;
 *              the caller keeps it unchanged in between (same desc, same
 *              inputs, the same conv_hist contents, so not one that
 *              conv_hist_out overwrote; the backward does not check this).
 *   workspace: 256-byte aligned, prism_forward_train_workspace() /
 *              prism_backward_train_workspace() bytes.
 * Errors: as for the plain entry points; a NULL, misaligned or too small
 * `saved` buffer gives PRISM_ERR_WORKSPACE / PRISM_ERR_ALIGN before any HIP
 * call. */
prism_status prism_saved_bytes(const prism_desc* desc, size_t* bytes);
prism_status prism_forward_train(const prism_desc* desc, const void* q, const void* k,
                                 const void* v, const float* alpha, const float* beta,
                                 const void* Wk, const void* Wp, const void* wbeta,
                                 const void* conv, const float* S0, const void* conv_hist,
                                 const int* cu_seqlens, void* o, float* ST, void* conv_hist_out,
                                 void* saved, size_t saved_bytes, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream);
prism_status prism_backward_train(const prism_desc* desc, const void* q, const void* k,
                                  const void* v, const float* alpha, const float* beta,
                                  const void* Wk, const void* Wp, const void* wbeta,
                                  const void* conv, const float* S0, const void* conv_hist,
                                  const int* cu_seqlens, const void* saved, size_t saved_bytes,
                                  const void* dO, const float* dST, void* dq, void* dk, void* dv,
                                  float* dalpha, float* dbeta, float* dWk, float* dWp,
                                  float* dwbeta, float* dconv, float* dS0, float* dconv_hist,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Recurrent form: the layer token by token (summary §2.1 S_t = S_{t-1} A_t
 * + B_t with §2.2's B_t, then o_t = S_t q_t), for the desc->T tokens of each
 * sequence in order.  With T = 1 this is the decode step of serving.
 *   S:          [B, H, dv, dk] f32, required, read as S_0 and overwritten
 *               with S_T (in place).
 *   conv_state: [B, 4, H, dv] dt, read as the ShortConv history before the
 *               tokens and overwritten with the history after them (in
 *               place); NULL means zeros, and nothing is written.
 *   o:          [B, T, H, dv] dt.
 *   workspace:  prism_step_workspace() bytes, 256-byte aligned (the
 *               refinement pairs of the tokens; 0 bytes and NULL allowed
 *               when L = 0).
 * The other inputs and desc fields are those of prism_forward; desc->chunk
 * must be valid but is not used.  A prism_forward over the first tokens
 * with ST and conv_hist_out, then prism_step over the rest, equals one
 * prism_forward over all of them up to rounding.  The state stays in
 * registers between tokens (one workgroup per sequence and head), so S
 * crosses HBM once per call.  Errors: as prism_forward. */
prism_status prism_step_workspace(const prism_desc* desc, size_t* bytes);
prism_status prism_step(const prism_desc* desc, const void* q, const void* k, const void* v,
                        const float* alpha, const float* beta, const void* Wk, const void* Wp,
                        const void* wbeta, const void* conv, float* S, void* conv_state, void* o,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);

/* prism_step without a workspace, for callers that cannot allocate device
 * memory (code under graph capture, tight serving loops, harnesses that
 * forbid allocation).  Same arguments, results and errors as prism_step,
 * except that the refinement pairs of the tokens go to a fixed device array
 * inside the library instead of a caller workspace:
 *   - the array holds 16 MiB per GPU (2 * B * H * L * T * dv elements of dt,
 *     each half rounded up to 256 bytes, must fit; e.g. B = 512, H = 16,
 *     L = 3, T = 1, dv = 128 in bf16); a larger call returns
 *     PRISM_ERR_WORKSPACE before any HIP call;
 *   - each GPU the library runs on keeps its own copy until the process
 *     ends; the call uses the copy of the device `stream` belongs to;
 *   - nothing is allocated or freed (no hipMalloc, hipFree or allocating
 *     library call): every pair the state kernel reads is written first by
 *     the same call, so the array needs no clearing between calls;
 *   - calls that overlap in time on one GPU (different streams, or several
 *     threads) share the array and race: serialise them. */
prism_status prism_step_noalloc(const prism_desc* desc, const void* q, const void* k,
                                const void* v, const float* alpha, const float* beta,
                                const void* Wk, const void* Wp, const void* wbeta,
                                const void* conv, float* S, void* conv_state, void* o,
                                hipStream_t stream);

/* ------------------------------------------------------------------------
 * Query / key normalisation with rotary positions
 * ------------------------------------------------------------------------
 * For every token and head, with x a row of d values (of q or of k):
 *   r = (c sum_i x_i^2 + eps)^(-1/2),  c = 1 (PRISM_NORM_L2) or 1/d (PRISM_NORM_RMS)
 *   y_i = x_i r w_i                    (w = wq or wk; NULL: ones)
 * and the first `rot` values of y turned in pairs by the token's position:
 *   (a, b) -> (a cos - b sin, b cos + a sin),  angle_i = 2 pi p turns[i] 2^-64,
 * pair i being (i, i + rot/2), or (2i, 2i + 1) with `interleaved`; the other
 * values pass.  turns[i] is the pair's frequency as an integer: turns per
 * position in units of 2^-64 (inv_freq / (2 pi) * 2^64, rounded).  The phase
 * p turns[i] mod 2^64 is formed exactly in integers, so the angle is as exact
 * at position 10^9 as at 1, with no table.  The arithmetic is fp32 (the sum of
 * squares too: rows of values beyond about 2^58, or without eps below about
 * 2^-58, leave its range); each output is rounded once to the storage type.
 * The outputs are what prism_forward and prism_linear_attention take as q
 * and k.                                                                   */
typedef enum {
  PRISM_NORM_L2 = 0,
  PRISM_NORM_RMS = 1,
  PRISM_NORM_LAYER = 2     /* mean and deviation, of prism_layer_norm alone */
} prism_norm;

/* Steps between consecutive batch entries, tokens and heads of a token
 * tensor, in elements (the last dimension is contiguous).                 */
typedef struct {
  long long batch, token, head;
} prism_strides;

/*   B, T       batch and tokens (>= 0; with B * T = 0 nothing is read)
 *   Hq, Hk     query and key heads (Hq >= 1, Hk >= 0; with Hk = 0 the key
 *              pointers are ignored)
 *   d          head dimension, a multiple of 8, 8 <= d <= 256
 *   rot        values of each head that are rotated: 0 or a multiple of 8,
 *              at most d; for 0, positions and turns are ignored
 *   eps        added under the root, finite and >= 0
 *   q, k       strides of the inputs; qo, ko: of the outputs (forward) or of
 *              their gradients (backward); dq, dk: of the input gradients
 *              (backward).  Multiples of 4 elements, magnitude < 2^40.      */
typedef struct {
  int B, T, Hq, Hk, d, rot;
  prism_dtype dtype;
  int norm;          /* PRISM_NORM_L2 or PRISM_NORM_RMS */
  int interleaved;   /* 0: pairs (i, i + rot/2), 1: pairs (2i, 2i + 1) */
  float eps;
  prism_strides q, k, qo, ko, dq, dk;
} prism_qk_norm_desc;

/* Forward.  q [B,T,Hq,d], k [B,T,Hk,d], qo, ko: dt, strided; wq, wk [d] dt or
 * NULL; positions [B,T] int32, contiguous (negative positions turn backwards);
 * turns [rot/2] int64.  qo may be q and ko may be k (same strides). */
prism_status prism_qk_norm(const prism_qk_norm_desc* desc, const void* q, const void* k,
                           const void* wq, const void* wk, const int* positions,
                           const long long* turns, void* qo, void* ko, hipStream_t stream);

/* Backward: gradients of <dqo, qo> + <dko, ko> from the forward's inputs (no
 * intermediate is kept).  With g = dy turned back by the angle, h = g w and
 * u = r x:  dx = r (h - c u (u . h)),   dw = sum over tokens and heads of g u.
 * dq, dk: dt, strided, written; dq may be dqo and dk may be dko.  dwq, dwk
 * [d] f32: written when wq / wk is given (required then, NULL otherwise).
 * The weight gradients are summed in a fixed order.  workspace:
 * prism_qk_norm_backward_workspace() bytes, 256-byte aligned (may be NULL
 * where that is 0: no weights). */
prism_status prism_qk_norm_backward_workspace(const prism_qk_norm_desc* desc, int weights,
                                              size_t* bytes);
prism_status prism_qk_norm_backward(const prism_qk_norm_desc* desc, const void* q, const void* k,
                                    const void* wq, const void* wk, const int* positions,
                                    const long long* turns, const void* dqo, const void* dko,
                                    void* dq, void* dk, float* dwq, float* dwk, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Linear attention with a decay for each head
 * ------------------------------------------------------------------------
 *   S_t = exp(g_t) S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
 * g is the log of the decay (f32): one number for each head, or one for each
 * token and head.  g = -inf (any g < -150, where exp underflows) forgets the
 * past.  The state has prism_forward's layout, [B, H, dv, dk] f32.
 * H query heads share Hk key / value heads: head h reads k, v of head
 * h / (H / Hk).  Chunks of tokens go through the matrix cores, with the state
 * between them carried in fp32.  In bf16, what a product adds to the state is
 * taken in three bf16 pieces where ST, dS0 or dg is wanted, so that these f32
 * results keep f32 accuracy, and in two where all results are bf16; the scaled
 * scores and the copy of the state that is read out are rounded once to bf16
 * (for dq and dk with dg: three pieces).  A bf16 o, dq, dk or dv is then off by
 * 2.4e-3 (2-norm, random values), where its own rounding alone gives 1.7e-3.
 * Sums of products (S, q . k v, S q, and the backward pass's own) below 2^76
 * (7e22) in magnitude never overflow on the way; larger ones may, although
 * their definition is still within fp32 (the step has no such limit).
 *
 *   B, H, Hk   sequences (>= 0), query heads, key / value heads (H % Hk = 0);
 *              B * H < 2^21
 *   T          tokens of each sequence (0 .. 2^30); packed: the longest length
 *   dk, dv     head dimensions, multiples of 16, 16 .. 128; H * dk, H * dv at
 *              most 2^22
 *   scale      finite
 *   packed_tokens  with cu_seqlens: rows N of the token tensors (the packed
 *              batches of prism_forward, sanitised the same way)
 *   q, k, v, o strides of q, k, v and of o / dO: multiples of 16 bytes, >= 0,
 *              a token step of at most 2^22 elements.  (packed: batch ignored)
 *   g          strides of g and dg in floats (>= 0); one decay for each head:
 *              batch = token = 0 (then dg is summed over batch and tokens;
 *              other zero steps that repeat a value are refused with dg)  */
typedef struct {
  int B, T, H, Hk, dk, dv;
  prism_dtype dtype;
  float scale;
  int packed_tokens;
  prism_strides q, k, v, o, g;
} prism_linear_attention_desc;

/* Workspace of the forward (backward = 0) or backward (1) pass, packed or
 * dense batch; with dg: of the backward pass that also gives dg.  The
 * workspace is 256-byte aligned, and may be NULL where 0 bytes are needed.
 * The first query serves both layouts, with room for the larger of B * T and
 * packed_tokens rows; the second the calls with cu_seqlens alone, with room
 * for packed_tokens rows (where lengths differ, far fewer than B * T). */
prism_status prism_linear_attention_workspace(const prism_linear_attention_desc* desc,
                                              int backward, int dg, size_t* bytes);
prism_status prism_linear_attention_packed_workspace(const prism_linear_attention_desc* desc,
                                                     int backward, int dg, size_t* bytes);

/* Whole sequences.  q [B,T,H,dk], k [B,T,Hk,dk], v [B,T,Hk,dv], o [B,T,H,dv]
 * dt, strided ([N,..] with cu_seqlens, B + 1 int32 offsets on the device);
 * S0 may be NULL (zeros); ST may be NULL, or S0 itself (updated in place).
 * A sequence of no tokens gives ST = S0.  A value that is not finite may
 * reach every row of its own sequence, never another sequence's. */
prism_status prism_linear_attention(const prism_linear_attention_desc* desc, const void* q,
                                    const void* k, const void* v, const float* g,
                                    const float* S0, const int* cu_seqlens, void* o, float* ST,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Gradients of <dO, o> + <dST, ST> from the forward's inputs.  dST may be
 * NULL (zeros).  dq [B,T,H,dk], dk [B,T,Hk,dk], dv [B,T,Hk,dv] dt,
 * contiguous; dg f32 (NULL: not wanted; zero where g < -104, whose decay is
 * zero; it is formed as a difference of sums over the tokens behind, good to
 * f32 against those sums: a dg_t far smaller than they are, as where exp(g_t)
 * is small, keeps fewer digits or none), dS0 f32 (NULL: not wanted; not the
 * buffer of dST or S0).  Written, not accumulated; packed rows outside every
 * (clamped) sequence are unspecified. */
prism_status prism_linear_attention_backward(const prism_linear_attention_desc* desc,
                                             const void* q, const void* k, const void* v,
                                             const float* g, const float* S0,
                                             const int* cu_seqlens, const void* dO,
                                             const float* dST, void* dq, void* dk, void* dv,
                                             float* dg, float* dS0, void* workspace,
                                             size_t workspace_bytes, hipStream_t stream);

/* The recurrence token by token, for the desc->T tokens of each sequence
 * (T = 1: a decode step): S is read as S_0, S_T goes to S_out (S_out = S:
 * in place).  T = 0 copies the state.  (Here as above, other outputs overlap
 * neither inputs nor one another.) */
prism_status prism_linear_attention_step(const prism_linear_attention_desc* desc, const void* q,
                                         const void* k, const void* v, const float* g,
                                         const float* S, float* S_out, void* o,
                                         hipStream_t stream);

/* ------------------------------------------------------------------------
 * Layer norm with the residual sum in front
 * ------------------------------------------------------------------------
 * For every row of D values (the width of the model, or of one head's output),
 *   s = x + residual,  m = mean(s)           (PRISM_NORM_RMS: m = 0)
 *   r = (mean((s - m)^2) + eps)^(-1/2),  y = (s - m) r w + b,  h = s.
 * The arithmetic is fp32; y is formed from the sum before it is rounded to the
 * storage type, which h then is.  The sum of a row's squared deviations has to be
 * within fp32's normal range: deviations below about 2^62 / sqrt(D), and, where eps
 * does not cover them, above about 2^-62.
 *
 * In this section and the following two, token tensors start at any multiple of
 * their element's size, and so do their rows; 16-byte rows are read faster.
 *
 *   B, T, H    rows: B * T * H of them, each >= 0, at most 2^30 in all
 *   D          values of a row, 1 .. 16384
 *   norm       PRISM_NORM_LAYER or PRISM_NORM_RMS
 *   eps        finite and >= 0
 *   x, r, y, h strides; r: of the residual (backward: of dh), y: of y (backward:
 *              of dy), h: of h (backward: of dx).  Magnitude < 2^40; of a
 *              result's dimensions of more than one entry each steps over all
 *              rows of those with smaller steps.                             */
typedef struct {
  int B, T, H, D;
  prism_dtype dtype;
  int norm;
  float eps;
  prism_strides x, r, y, h;
} prism_layer_norm_desc;

/* Forward.  x, residual, y, h [B,T,H,D] dt, strided; w, b [D] dt or NULL (ones,
 * zeros).  residual may be NULL (s = x; h is then NULL too); h may be NULL (the
 * sum is not wanted).  y and h may each be x or residual, with its strides, but
 * not each other. */
prism_status prism_layer_norm(const prism_layer_norm_desc* desc, const void* x,
                              const void* residual, const void* w, const void* b, void* y, void* h,
                              hipStream_t stream);

/* Backward, from x, the rows that were normalised (h where there was a
 * residual): with u = (x - m) r and g = dy w,
 *   dx = r (g - mean(g) - u mean(g u)) + dh   (PRISM_NORM_RMS: without mean(g))
 *   dw = sum over rows of dy u,  db = sum over rows of dy.
 * dh, the gradient that reaches the sum by itself, may be NULL (zero); dx, dt,
 * is the gradient of x and of the residual alike, and may be dy, dh or x.
 * dw, db [D] f32: NULL where not wanted; summed in a fixed order.  workspace:
 * prism_layer_norm_backward_workspace() bytes (weights: whether dw or db is
 * wanted), 256-byte aligned (may be NULL where that is 0). */
prism_status prism_layer_norm_backward_workspace(const prism_layer_norm_desc* desc, int weights,
                                                 size_t* bytes);
prism_status prism_layer_norm_backward(const prism_layer_norm_desc* desc, const void* x,
                                       const void* w, const void* dy, const void* dh, void* dx,
                                       float* dw, float* db, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Short convolution
 * ------------------------------------------------------------------------
 * The depthwise causal convolution by itself (the layer's anchor has it on v):
 * for every channel,
 *   z_t = b + sum_{j < K} w[c, j] x_{t-j},  y_t = z_t (PRISM_ACT_IDENTITY) or
 *   z_t sigmoid(z_t) (PRISM_ACT_SILU),
 * x_{-1}, x_{-2}, .. from hist.  The arithmetic is fp32, y rounded once.
 *
 *   B, T, D    sequences, tokens (each >= 0, at most 2^30 tokens in all), channels
 *              (1 .. 4194304); B * D < 2^31 and B * ceil(D / 256) < 2^23
 *   K          taps, 2 .. 4
 *   activation PRISM_ACT_IDENTITY or PRISM_ACT_SILU
 *   packed_tokens  with cu_seqlens: rows N of the token tensors (T is then not
 *              used).  Offsets as in prism_forward's packed batches, clamped the
 *              same way; a sequence is as long as they say, and rows of no
 *              sequence stay as they are.
 *   x, y, dx   strides (batch and token; head is not used) of x, of y (backward:
 *              of dy) and, backward, of dx, as in prism_layer_norm_desc      */
typedef struct {
  int B, T, D, K;
  prism_dtype dtype;
  int activation;
  int packed_tokens;
  prism_strides x, y, dx;
} prism_short_conv_desc;

/* Forward.  x, y [B,T,D] ([N,D] with cu_seqlens) dt, strided; w [D,K] dt, tap j
 * multiplying x_{t-j}; b [D] dt or NULL; hist [B,K-1,D] dt, the tokens before the
 * sequence, oldest first, or NULL (zeros); hist_out (may be NULL) receives the
 * last K - 1 tokens for the next call, from hist or zeros where the sequence is
 * shorter, and may be hist itself.  Apart from that no result overlaps an input or
 * the other result. */
prism_status prism_short_conv(const prism_short_conv_desc* desc, const void* x, const void* w,
                              const void* b, const void* hist, const int* cu_seqlens, void* y,
                              void* hist_out, hipStream_t stream);

/* Backward: gradients of <dy, y> from the forward's inputs (hist as the forward
 * read it).  dx dt, strided; dw [D,K] f32; db [D] f32 or NULL; dhist [B,K-1,D] f32
 * or NULL (add it to the last rows of the gradient of the call before).  Written,
 * not accumulated; the sums over tokens in a fixed order.  workspace:
 * prism_short_conv_backward_workspace() bytes (packed: whether cu_seqlens is
 * given), 256-byte aligned.  No output overlaps an input. */
prism_status prism_short_conv_backward_workspace(const prism_short_conv_desc* desc, int packed,
                                                 size_t* bytes);
prism_status prism_short_conv_backward(const prism_short_conv_desc* desc, const void* x,
                                       const void* w, const void* b, const void* hist,
                                       const int* cu_seqlens, const void* dy, void* dx, float* dw,
                                       float* db, float* dhist, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------------
 * Gated recurrence
 * ------------------------------------------------------------------------
 * A state of one value a channel: h_t = a_t h_{t-1} + u_t with the gates formed
 * in the same pass.  With s = sigmoid(i), or 1 without i,
 *   PRISM_GATE_LOG      a = exp(f),                  u = s x
 *   PRISM_GATE_SIGMOID  a = sigmoid(f),              u = (1 - a) s x
 *   PRISM_GATE_POWER    a = exp(-lam sigmoid(f)),    u = sqrt(1 - a^2) s x
 * lam [D] f32, >= 0.  f of PRISM_GATE_LOG is at most 0 in earnest; above it, the
 * product of the decays of any 128 tokens in a row has to stay within fp32.
 * Gates, state and sums are fp32 (1 - a and 1 - a^2 to their own size; of numbers
 * below 2^-126, the forward pass may take 1 - a^2 and both may take sigmoid(f) as
 * 0); h is rounded once.  A value that is not finite may reach every later token of
 * its sequence and channel, never another's, or be forgotten where the decays since
 * then multiply to 0 in fp32.
 *
 *   B, T, D    as in prism_short_conv_desc, and, of N tokens in all,
 *              ceil(N / 64) * ceil(D / 64) <= 2^22
 *   gate       a prism_gate value
 *   packed_tokens  as in prism_short_conv_desc
 *   x, f, i, h strides (batch and token) of the inputs and of h; dh, dx, df, di:
 *              backward, as in prism_layer_norm_desc                         */
typedef enum {
  PRISM_GATE_LOG = 0,
  PRISM_GATE_SIGMOID = 1,
  PRISM_GATE_POWER = 2
} prism_gate;
typedef struct {
  int B, T, D;
  prism_dtype dtype;
  int gate;
  int packed_tokens;
  prism_strides x, f, i, h, dh, dx, df, di;
} prism_gated_recurrence_desc;

/* Workspace of the forward (backward = 0) or backward (1) pass, of a packed
 * batch or a dense one; 256-byte aligned, may be NULL where 0 bytes are needed.
 * Passes in flight at the same time need one each. */
prism_status prism_gated_recurrence_workspace(const prism_gated_recurrence_desc* desc, int packed,
                                              int backward, size_t* bytes);

/* Whole sequences.  x, f, i, h [B,T,D] ([N,D] with cu_seqlens) dt, strided; i may
 * be NULL; lam is NULL but with PRISM_GATE_POWER.  h0 [B,D] f32, the state before
 * the sequence, may be NULL (zeros); hT [B,D] f32, the state after it, may be NULL,
 * or h0 itself.  A sequence of no tokens gives hT = h0.  Apart from that no result
 * overlaps an input or the other result. */
prism_status prism_gated_recurrence(const prism_gated_recurrence_desc* desc, const void* x,
                                    const void* f, const void* i, const float* lam,
                                    const float* h0, const int* cu_seqlens, void* h, float* hT,
                                    void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Gradients of <dh, h> + <dhT, hT> from the forward's inputs and its output h,
 * which is read as h_{t-1} (in bf16 as rounded: df and dlam then carry its
 * rounding, of at most 2^-8 of each h_{t-1}).  dhT [B,D] f32 may be NULL (zero).
 * dx, df, di dt, strided (di: NULL without i); dlam [D] f32, NULL but with
 * PRISM_GATE_POWER, summed in a fixed order; dh0 [B,D] f32 or NULL (not the buffer
 * of dhT or h0).  Where lam or sigmoid(f) is 0 the root's infinite slope is taken as 0.
 * Written, not accumulated; no result overlaps an input or another result. */
prism_status prism_gated_recurrence_backward(const prism_gated_recurrence_desc* desc,
                                             const void* x, const void* f, const void* i,
                                             const float* lam, const float* h0,
                                             const int* cu_seqlens, const void* h, const void* dh,
                                             const float* dhT, void* dx, void* df, void* di,
                                             float* dlam, float* dh0, void* workspace,
                                             size_t workspace_bytes, hipStream_t stream);

/* Token by token for the T tokens of each dense sequence (T = 1: a decode step):
 * state [B,D] f32 is read, the state after the tokens goes to state_out (state
 * itself: in place).  Apart from that no result overlaps an input. */
prism_status prism_gated_recurrence_step(const prism_gated_recurrence_desc* desc, const void* x,
                                         const void* f, const void* i, const float* lam,
                                         const float* state, float* state_out, void* h,
                                         hipStream_t stream);

/* Human-readable name of a status code (static string). */
const char* prism_status_string(prism_status status);

/* Detail of the last failure on the calling thread ("" if none). */
const char* prism_last_error(void);

/* Kernel timing.  Between prism_timing_begin() and prism_timing_end(), every
 * kernel the library enqueues is bracketed by two HIP events recorded on the
 * stream it runs on.  prism_timing_end() waits for those events and fills up
 * to `capacity` entries: names[i] (static strings), total_ms[i] (sum of the
 * event-measured durations) and launches[i]; it returns the number of
 * distinct kernels.  Not thread-safe; meant for benchmarks. */
void prism_timing_begin(void);
int prism_timing_end(const char** names, double* total_ms, int* launches, int capacity);

#ifdef __cplusplus
}
#endif

#endif /* PRISM_H_ */
