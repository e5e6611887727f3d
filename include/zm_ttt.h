/*
 * zm_ttt.h - C ABI of the large-chunk test-time-training (TTT) layer for
 * AMD Instinct MI355X (gfx950).
 *
 * The layer keeps, per head, a SwiGLU fast weight
 *     f_W(x) = W2 [ SiLU(W1 x) (*) (W3 x) ]          (elementwise product (*))
 * with W1, W3 of shape [h, d] and W2 of shape [d, h].  An update takes one
 * gradient step on the virtual loss  -sum_i eta_i f_W(k_i)^T v_i  summed over
 * every token of a chunk, optionally renormalises each row of the updated
 * weights to its pre-update L2 norm, and an apply reads queries through the
 * weights.
 *   Sources: "[논문리뷰] ZipMap: Linear-Time Stateful 3D Reconstruction via
 *   Test-Time Training" (kimjy99.github.io), Method 2. Feature Backbone,
 *   Eq. (1) (SwiGLU), Eq. (2) (loss), Eq. (3) (chunk gradient with per-token
 *   rate), the renormalised update display, Eq. (4) (apply), and 3. Streaming
 *   Reconstruction, Eq. (6); the ZipMap paper-reading notes (67656.sbs),
 *   sections on Eq. 2 / Eq. 3 and streaming; the mhpn.cn LaCT summary, part
 *   2、架构 (gradients summed over the whole chunk, L2 normalisation) and
 *   3、应用场景 (apply/update orders).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Memory: every pointer is device memory owned by the caller.  The library
 *    allocates nothing, keeps no state between calls (apart from the optional
 *    profiling events below) and never synchronises the stream.  Exception:
 *    the full-width shape (d_head 1024, d_hidden 2048) runs its dense products
 *    through hipBLASLt, whose handle the library creates on the first such
 *    call on a device (the GEMM library then holds its own resources until the
 *    process ends) and whose chosen algorithm per problem shape it caches.
 *  - Token tensors q, k, v, o: [n, heads, d_head] with a token stride of
 *    desc->ld_tok elements (heads * d_head <= ld_tok <= 2^24, multiple of 8;
 *    a larger stride is rejected with ZM_ERR_INVALID_ARG).  Element
 *    type: bf16 or fp32 (desc->io_dtype).  Base pointers 16-byte aligned.
 *  - eta: fp32 [n, heads], contiguous (token-major), 4-byte aligned.
 *  - Weights: fp32, contiguous, 16-byte aligned; W1 and W3 [heads, h, d],
 *    W2 [heads, d, h].  The weights are always fp32; with bf16 io the kernels
 *    round them to bf16 operands and accumulate in fp32.
 *  - Workspace: device scratch of at least zm_ttt_workspace_size() bytes,
 *    256-byte aligned.  Calls sharing one workspace must not overlap in time;
 *    calls on distinct workspaces and streams are independent.  For short
 *    chunks (bf16 io, heads a multiple of 8, the gradient step) an update
 *    reduces its partial sums inside its own launch, whose workgroups meet
 *    at counters kept in the workspace; should that ever fail (a wait past
 *    its 2 s bound), the stepped weights come out NaN, never plausible wrong
 *    values.
 *  - stream: a hipStream_t passed as void*; NULL is the default stream.
 *    Every entry point only enqueues work and returns.
 *  - Errors: arguments are checked on the host before any HIP call; a failed
 *    check returns a negative zm_status and enqueues nothing.  A failed
 *    launch returns ZM_ERR_HIP.  Faults inside kernels surface at the
 *    caller's next synchronisation.  NaN/Inf inputs propagate (one NaN token
 *    poisons the chunk sum); they are not checked.
 *  - Supported shapes: (d_head, d_hidden) in {(64,128), (64,256), (128,128),
 *    (128,256)}, and the full-width (1024, 2048) with bf16 io (the ZipMap
 *    notes' single full-width fast weight with a 6 d^2 state, d = 1024);
 *    heads in [1, 64]; others return ZM_ERR_UNSUPPORTED.
 *  - Results are deterministic: the split of the token sum depends only on
 *    (n, heads, d_head, d_hidden), and partial sums are combined in a fixed
 *    order without atomics.
 */
#ifndef ZM_TTT_H
#define ZM_TTT_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__) || defined(__clang__)
#define ZM_API __attribute__((visibility("default")))
#else
#define ZM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Size of the device scratch array behind zm_ttt_update_apply_scratch. */
#define ZM_TTT_SCRATCH_BYTES ((size_t)64 << 20)

typedef enum zm_status {
  ZM_OK = 0,
  ZM_ERR_INVALID_ARG = -1,   /* null/misaligned pointer, bad size or enum */
  ZM_ERR_UNSUPPORTED = -2,   /* valid but unsupported shape */
  ZM_ERR_WORKSPACE = -3,     /* workspace missing or too small */
  ZM_ERR_HIP = -4            /* a HIP launch or runtime call failed */
} zm_status;

typedef enum zm_dtype { ZM_BF16 = 0, ZM_F32 = 1 } zm_dtype;

/* Row renormalisation after the step: each row r (the fan-in vector of one
 * output unit: a row of W1 or W3 of length d, a row of W2 of length h) is
 * rescaled to ||W_r|| / max(||W'_r||, 1e-12) times itself, ||W_r|| being the
 * norm before the update (review, renormalised update display). */
typedef enum zm_renorm { ZM_RENORM_NONE = 0, ZM_RENORM_ROW = 1 } zm_renorm;

/* Per-frame order of the streaming step (LaCT summary, 3、应用场景):
 * APPLY_THEN_UPDATE reads frame t with W(t-1) and then writes it;
 * UPDATE_THEN_APPLY writes frame t first and reads it with W(t). */
typedef enum zm_order { ZM_APPLY_THEN_UPDATE = 0, ZM_UPDATE_THEN_APPLY = 1 } zm_order;

/* Flags OR-ed into the order argument of zm_ttt_stream_step, for a caller that
 * streams frames through one workspace: the bf16 operand copies of W that a
 * frame's reduce writes serve the next frame, which then skips its separate
 * rounding launch (bf16 io; with fp32 io the flags have no effect):
 *   ZM_STREAM_EMIT_BF16:  on return the workspace holds the bf16 operand
 *     copies of the state the call leaves in w1, w2, w3;
 *   ZM_STREAM_REUSE_BF16: the workspace already holds the bf16 operand copies
 *     of the incoming state, left by the previous call on this workspace with
 *     ZM_STREAM_EMIT_BF16; the call does not round w1, w2, w3 again.
 * A stream passes EMIT on its first frame and EMIT | REUSE on the others.
 * With REUSE the caller guarantees that since that previous call neither the
 * workspace nor w1, w2, w3 changed and the descriptor is the same; otherwise
 * the results are undefined (the library keeps no state to check it).  The
 * results are bitwise those of calls without the flags. */
typedef enum zm_stream_flags {
  ZM_STREAM_EMIT_BF16 = 0x100,
  ZM_STREAM_REUSE_BF16 = 0x200
} zm_stream_flags;

/* The step taken with the chunk gradient g of one weight matrix (review, the
 * update display after Eq. (3)):
 *   ZM_STEP_GRADIENT:      W' = W - g;
 *   ZM_STEP_NEWTON_SCHULZ: W' = W - NewtonSchulz(g), the orthonormalisation of
 *     the Muon optimizer that the review names.  The pages give neither its
 *     polynomial nor its step count; the library runs Muon's published odd
 *     quintic: five steps of X <- a X + b (X X^T) X + c (X X^T)^2 X with
 *     (a, b, c) = (3.4445, -4.7750, 2.0315) from X = g / max(||g||_F, 1e-12),
 *     per head and per matrix.  Its products run in split-bf16 (hi + lo
 *     parts, three bf16 matrix-core products each, fp32 accumulation) with bf16
 *     io and in fp32 with fp32 io (at the full-width shape as batched library
 *     GEMMs, three per product).  The result no longer scales with eta: the
 *     step has singular values near 1 whatever the gradient's size, so it is
 *     meant to be used with ZM_RENORM_ROW.  n_kv = 0 leaves W unchanged. */
typedef enum zm_step_rule { ZM_STEP_GRADIENT = 0, ZM_STEP_NEWTON_SCHULZ = 1 } zm_step_rule;

typedef struct zm_ttt_desc {
  int32_t heads;      /* independent fast weights */
  int32_t d_head;     /* d: width of q, k, v, o per head */
  int32_t d_hidden;   /* h: SwiGLU hidden width */
  int32_t io_dtype;   /* zm_dtype of q, k, v, o */
  int32_t renorm;     /* zm_renorm */
  int32_t step_rule;  /* zm_step_rule (0: plain gradient step) */
  int64_t ld_tok;     /* elements between consecutive tokens of q/k/v/o */
} zm_ttt_desc;

/* Bytes of workspace needed by any entry point below for an update over
 * n_kv tokens and an apply over n_q queries (either may be 0).  Writes the
 * size to *bytes.  Returns ZM_OK or a validation error.  The size never
 * decreases as n_kv or n_q grows, so a workspace sized for (n_kv, n_q) also
 * serves every call over at most n_kv tokens and n_q queries. */
ZM_API int zm_ttt_workspace_size(const zm_ttt_desc* desc, int64_t n_kv, int64_t n_q, size_t* bytes);

/* Update (review Eq. (2)-(3) and the renormalised update display):
 *   g = grad_W sum_{i<n_kv} eta_i L(f_W(k_i), v_i),  L(f, v) = -f^T v,
 *   W' = W - g  (or W - NewtonSchulz(g), see zm_step_rule),
 *   W_hat = renorm(W, W') if desc->renorm else W'.
 * k, v: [n_kv, heads, d_head] tokens; eta: [n_kv, heads].
 * w1, w2, w3: the current fast weights (read only).
 * w1_out, w2_out, w3_out: receive W_hat; they may alias w1, w2, w3 (in-place
 * update).  n_kv = 0 is valid and gives W_hat = W. */
ZM_API int zm_ttt_update(const zm_ttt_desc* desc, int64_t n_kv,
                  const void* k, const void* v, const float* eta,
                  const float* w1, const float* w2, const float* w3,
                  float* w1_out, float* w2_out, float* w3_out,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Update and its virtual loss (review Eq. (2)): as zm_ttt_update, and
 * loss[h] = sum_{i<n_kv} eta_i L(f_W(k_i), v_i) = -sum_i eta_i f_W(k_i)^T v_i
 * of head h at the incoming W (the loss whose gradient the step follows).
 * It is read from the update's own registers: f^T v = u . (W2^T v) with
 * u = SiLU(W1 k) (*) W3 k and W2^T v both formed for the gradient, so the
 * loss costs one multiply-add per (token, hidden unit) and a fixed-order
 * sum.  loss: device pointer to heads floats (fp32; operands as the update's
 * bf16 ones).  n_kv = 0 writes zeros.  Bitwise reproducible; W_hat is
 * bitwise that of zm_ttt_update.  The bf16 narrow heads only: fp32 io and the
 * full-width shape return ZM_ERR_UNSUPPORTED.  Workspace as zm_ttt_update. */
ZM_API int zm_ttt_update_loss(const zm_ttt_desc* desc, int64_t n_kv,
                  const void* k, const void* v, const float* eta,
                  const float* w1, const float* w2, const float* w3,
                  float* w1_out, float* w2_out, float* w3_out, float* loss,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Apply (review Eq. (4)): o_i = f_W(q_i) for i < n_q, per head.
 * q, o: [n_q, heads, d_head] in desc->io_dtype; o must not overlap q. */
ZM_API int zm_ttt_apply(const zm_ttt_desc* desc, int64_t n_q, const void* q,
                 const float* w1, const float* w2, const float* w3,
                 void* o, void* workspace, size_t workspace_bytes, void* stream);

/* Bidirectional single chunk (review of ZipMap, Method 2: the chunk update of
 * Eq. (3) over all image tokens, then the read of Eq. (4) with the updated
 * weights; the ZipMap notes' TTT-module section describes the same write-then-
 * read of one chunk; a ray-map target view only reads): the update over all
 * n_kv tokens, then the apply of all n_q queries through W_hat (the queries
 * may include extra target-view rows beyond the image tokens).  Outputs W_hat
 * to w*_out (may alias w*) and o.  Equivalent to zm_ttt_update followed by
 * zm_ttt_apply on W_hat, without re-reading W_hat from fp32. */
ZM_API int zm_ttt_update_apply(const zm_ttt_desc* desc, int64_t n_kv,
                        const void* k, const void* v, const float* eta,
                        int64_t n_q, const void* q,
                        const float* w1, const float* w2, const float* w3,
                        float* w1_out, float* w2_out, float* w3_out, void* o,
                        void* workspace, size_t workspace_bytes, void* stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * update and apply as zm_ttt_update_apply, run in a scratch array the library
 * holds in device memory (ZM_TTT_SCRATCH_BYTES = 64 MiB, one copy per GPU
 * from module load to process end) instead of a caller workspace.  The
 * call allocates nothing; on its first use on a device it looks up that
 * device's scratch address.  Results are bitwise those of
 * zm_ttt_update_apply.  Narrow heads only: a call whose workspace need
 * (zm_ttt_workspace_size(desc, n_kv, n_q)) exceeds the scratch returns
 * ZM_ERR_WORKSPACE, and the full-width shape ZM_ERR_UNSUPPORTED.  Every
 * kernel writes what the next one reads, except the counters of the
 * in-launch reduce (see Workspace above), which must start at zero: the
 * call's first kernel clears them (a kernel, not a memset, so the call can
 * be captured).  A call leaves its last contents there.  All calls on one GPU share its
 * scratch: calls that overlap in time on one GPU (two streams, two threads)
 * race and give undefined results; order them on one stream. */
ZM_API int zm_ttt_update_apply_scratch(const zm_ttt_desc* desc, int64_t n_kv,
                                const void* k, const void* v, const float* eta,
                                int64_t n_q, const void* q,
                                const float* w1, const float* w2, const float* w3,
                                float* w1_out, float* w2_out, float* w3_out, void* o,
                                void* stream);

/* One streaming step on one frame of n_frame tokens (review 3. Streaming
 * Reconstruction, Eq. (6)).  order: a zm_order, optionally OR-ed with
 * zm_stream_flags.  w1, w2, w3 hold the state W(t-1) on entry and
 * W(t) on return (updated in place).  q, k, v: [n_frame, heads, d_head];
 * eta: [n_frame, heads]; o receives f_{W(t-1)}(q) (APPLY_THEN_UPDATE) or
 * f_{W(t)}(q) (UPDATE_THEN_APPLY).  o must not overlap q, k, v or eta: with
 * APPLY_THEN_UPDATE and bf16 io the read and the update's partial sums run
 * side by side in one launch. */
ZM_API int zm_ttt_stream_step(const zm_ttt_desc* desc, int order, int64_t n_frame,
                       const void* q, const void* k, const void* v, const float* eta,
                       float* w1, float* w2, float* w3, void* o,
                       void* workspace, size_t workspace_bytes, void* stream);

/* A sequence of n = offsets[n_chunks] tokens cut into consecutive chunks
 * [offsets[c], offsets[c+1]), read and written chunk after chunk with the
 * orders of the LaCT summary (mhpn.cn, part 二, 3、应用场景):
 *   ZM_UPDATE_THEN_APPLY: block-causal, W <- Update(W; chunk c), then
 *     o_c = f_W(q_c) (order (b));
 *   ZM_APPLY_THEN_UPDATE: shifted block-causal, o_c = f_W(q_c), then
 *     W <- Update(W; chunk c) (order (c)).
 * update_mask (host memory, n_chunks bytes, or NULL for all): a zero entry
 * skips chunk c's update, so that chunk is only read (updates on selected
 * chunks and reads on all, order (d)).  inner_steps (1..64) repeats the
 * update on the same chunk, each step taking the gradient at the weights the
 * previous one produced.  A per-chunk rate is a scaling of that chunk's eta
 * rows.
 * offsets: host memory, n_chunks + 1 int64, offsets[0] = 0, non-decreasing;
 * n_chunks in [0, 2^24].  Empty chunks are skipped.
 * q, k, v, o: [n, heads, d_head]; eta: [n, heads]; o must not overlap q, k,
 * v or eta (as for zm_ttt_stream_step).  w1, w2, w3 hold the state and are
 * updated in place.  The workspace must hold
 * zm_ttt_workspace_size(desc, L, L) bytes, L the longest chunk.  Equivalent to
 * one zm_ttt_stream_step per chunk (extended by the mask and inner steps). */
ZM_API int zm_ttt_chunked(const zm_ttt_desc* desc, int order, int64_t n_chunks,
                   const int64_t* offsets, const uint8_t* update_mask, int inner_steps,
                   const void* q, const void* k, const void* v, const float* eta,
                   float* w1, float* w2, float* w3, void* o,
                   void* workspace, size_t workspace_bytes, void* stream);

/* Layer norm of token rows, as in front of zm_ttt_layer's projections:
 *   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) r gamma + beta
 * over the width of each row, in fp32 (the variance from the distances to the
 * mean), rounded once to the io type. */
typedef struct zm_norm_desc {
  int32_t width;      /* a multiple of 8, at most 8192 (wider: ZM_ERR_UNSUPPORTED) */
  int32_t io_dtype;   /* zm_dtype of x, y, dy, dx */
  float eps;          /* > 0 */
  int32_t reserved;   /* must be 0 */
} zm_norm_desc;

/* x, y: [n][width] rows of strides ld_x, ld_y (>= width, multiples of 8), bases
 * 16-byte aligned.  gamma, beta: fp32 [width], 16-byte aligned, either may be NULL (1, 0).
 * stats: NULL, or fp32 [2][n] that receives mu, then r, for the backward.  y
 * may be x (same stride); otherwise they must not overlap.  n = 0 is valid. */
ZM_API int zm_layer_norm(const zm_norm_desc* desc, int64_t n, const void* x, int64_t ld_x,
                  const float* gamma, const float* beta, void* y, int64_t ld_y, float* stats,
                  void* stream);

/* Bytes of workspace of zm_layer_norm_backward (never less for more rows). */
ZM_API int zm_layer_norm_backward_workspace_size(const zm_norm_desc* desc, int64_t n, size_t* bytes);

/* The gradient: with xh = (x - mu) r from stats and a = dy gamma,
 *   dx = r (a - mean(a) - xh mean(a xh)), dgamma = sum_rows dy xh, dbeta = sum_rows dy.
 * dgamma, dbeta: fp32 [width], overwritten (n = 0: zeros); either may be NULL, and they
 * must not be one array (refused).
 * dx may be dy or x (same stride).  Sums in fixed order: bitwise reproducible.
 * The workspace is 256-byte aligned; with both dgamma and dbeta NULL it is not
 * read and may be NULL. */
ZM_API int zm_layer_norm_backward(const zm_norm_desc* desc, int64_t n, const void* dy, int64_t ld_dy,
                  const void* x, int64_t ld_x, const float* gamma, const float* stats,
                  void* dx, int64_t ld_dx, float* dgamma, float* dbeta,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Rotary positions with up to four axes (time, height, width) on the q and k of
 * [n, heads, d_head] tokens.  Pair p < P = sum of sections belongs to the axis
 * whose section holds it (axis 0's pairs first) and turns by the angle
 * pos[t][axis] freqs[p]:  (x, y) -> (x cos - y sin, x sin + y cos).
 * The two dims of pair p:
 *   ZM_ROTARY_HALVES       p and p + P
 *   ZM_ROTARY_PAIRS        2 p and 2 p + 1
 *   ZM_ROTARY_AXIS_HALVES  the halves of the axis's own block: with f the pairs
 *                          of earlier axes and s its own, p + f and p + f + s
 * Dims from 2 P on pass unrotated.  Cosine and sine are those of the angle in 64
 * bits, so far positions lose no precision; position 0 (as of
 * a frame's special tokens) leaves finite values unchanged.  A position that is
 * infinite or NaN gives NaN in the pairs of its axis. */
typedef enum zm_rotary_layout {
  ZM_ROTARY_HALVES = 0,
  ZM_ROTARY_PAIRS = 1,
  ZM_ROTARY_AXIS_HALVES = 2
} zm_rotary_layout;

typedef struct zm_rotary_desc {
  int32_t heads_q;      /* 1..64 */
  int32_t heads_k;      /* 0..64; 0: no k, its pointers are not read */
  int32_t d_head;       /* a multiple of 8, at most 256 (wider: ZM_ERR_UNSUPPORTED) */
  int32_t io_dtype;     /* zm_dtype of q, k */
  int32_t layout;       /* zm_rotary_layout */
  int32_t inverse;      /* 0, or 1: by minus the angle (the rotation's gradient) */
  int32_t pos_f32;      /* positions: 0 int32, 1 fp32 */
  int32_t axes;         /* 1..4 */
  int32_t sections[4];  /* pairs of each axis, >= 0; 1 <= P <= d_head / 2; unused axes 0 */
  int64_t ld_q, ld_k, ld_q_out, ld_k_out;  /* token strides, multiples of 8, >= heads * d_head */
} zm_rotary_desc;

/* pos: [n][axes] contiguous; freqs: fp32 [P] (radians per unit of position).
 * q_out may be q and k_out may be k (same stride: in place, what is unrotated
 * keeps its bits); otherwise an output must not overlap another array (k's
 * pointer for q_out, q's for k_out or one for both is refused).  q and k
 * may be slices of one projection's rows.  n = 0 is valid. */
ZM_API int zm_rotary(const zm_rotary_desc* desc, int64_t n, const void* pos, const float* freqs,
              const void* q, const void* k, void* q_out, void* k_out, void* stream);

/* The heads of q and k normalised and rotated in one pass: per head x of d_head elements
 *   y = rotate((x - mu) / sqrt(mean((x - mu)^2) + eps) gamma + beta),
 * mu = mean(x) (ZM_NORM_LAYER) or 0 (ZM_NORM_RMS), statistics in fp32 (elements below 2^60 in
 * size), one rounding at the end, the rotation as zm_rotary's (rotary.inverse must be 0). */
typedef enum zm_norm_kind { ZM_NORM_RMS = 0, ZM_NORM_LAYER = 1 } zm_norm_kind;

typedef struct zm_norm_rotary_desc {
  zm_rotary_desc rotary;
  int32_t norm;         /* zm_norm_kind */
  float eps;            /* > 0 */
} zm_norm_rotary_desc;

/* Arrays as for zm_rotary; gammas and betas: fp32 [d_head], 16-byte aligned, or NULL (ones,
 * zeros), the same for every head of their tensor. */
ZM_API int zm_norm_rotary(const zm_norm_rotary_desc* desc, int64_t n, const void* pos, const float* freqs,
              const void* q, const void* k, const float* q_gamma, const float* q_beta,
              const float* k_gamma, const float* k_beta, void* q_out, void* k_out, void* stream);

/* Bytes of workspace of zm_norm_rotary_backward (16 KB a head dim at most; never less for more tokens). */
ZM_API int zm_norm_rotary_backward_workspace_size(const zm_norm_rotary_desc* desc, int64_t n, size_t* bytes);

/* The gradient from the inputs: dq_out, dk_out, the gradients of q_out, k_out (strides
 * rotary.ld_q_out, ld_k_out), give dq, dk (the io type) and, fp32 [d_head], summed over tokens
 * and heads, the parameters' gradients (each NULL: not wanted; without k's heads zeros).
 * dq may be dq_out or q (same stride), dk dk_out or k; otherwise the outputs must not overlap
 * other arrays.  Bitwise reproducible.  The workspace is needed with a parameter's gradient and n > 0. */
ZM_API int zm_norm_rotary_backward(const zm_norm_rotary_desc* desc, int64_t n, const void* pos, const float* freqs,
              const void* dq_out, const void* dk_out, const void* q, const void* k,
              const float* q_gamma, const float* k_gamma,
              void* dq, int64_t ld_dq, void* dk, int64_t ld_dk,
              float* dq_gamma, float* dq_beta, float* dk_gamma, float* dk_beta,
              void* workspace, size_t workspace_bytes, void* stream);

/* Gated delta rule: the linear fast weight f_S(x) = S x, S [d_head][d_head] fp32
 * per value head, trained token by token on |S k - v|^2 / 2 with a decay
 * (the notes' linear case of the fast weight, with one gradient step of rate
 * beta_t to each token instead of one to a chunk, and a gate):
 *   S_t = a_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,  a_t = exp(g_t),
 *   o_t = scale S_t q_t.
 * Tokens: q, k [n, heads_k, d_head], v, o [n, heads, d_head] (value head h reads
 * key head h / (heads / heads_k)); g (log decay, any value; -inf resets the
 * state) and beta fp32 [n, heads] contiguous.  Keys are used as they are: the
 * recurrence contracts for beta |k|^2 in [0, 2].
 * Sequences lie one after the other: sequence b has the tokens offsets[b] ..
 * offsets[b + 1] - 1 (device int32 [n_seq + 1], nondecreasing in 0..n; values
 * outside are clamped to that), which may be none.  offsets may be NULL for a
 * single sequence of all n tokens.  Rows of the outputs outside every sequence
 * are left as they were.  A token that is not finite can make NaN, in its heads, of
 * the outputs of the 64 tokens that it is taken with (counted from its sequence's
 * first) and of later ones and of its sequence's gradients; earlier chunks'
 * outputs and other sequences stay as they are.
 * Values of tokens and states stay below 2^60 in size (they are scaled by up to that); where
 * positive g make a state grow, tokens' values under 2^-40 may lose bits to the same scaling.
 * States: fp32 [n_seq, heads, d_head (rows: v), d_head (k)], 16-byte aligned. */
typedef struct zm_delta_desc {
  int32_t heads;      /* value heads, 1..64, a multiple of heads_k */
  int32_t heads_k;    /* query/key heads */
  int32_t d_head;     /* 64 or 128 */
  int32_t io_dtype;   /* zm_dtype of q, k, v, o and their gradients */
  int32_t n_seq;      /* sequences, >= 0 */
  float scale;        /* of the outputs */
  int64_t ld_q, ld_k, ld_v, ld_o;  /* token strides: >= heads * d_head (q, k: heads_k *
                                      d_head), multiples of 8, at most 2^24 */
} zm_delta_desc;

/* Bytes of workspace of zm_delta_rule for n tokens in desc->n_seq sequences (never less for
 * more tokens). */
ZM_API int zm_delta_rule_workspace_size(const zm_delta_desc* desc, int64_t n, size_t* bytes);

/* The rule over whole sequences, 64 tokens at a time (fp32 states, products of
 * 24 bits up to a state and up to an output's own rounding).  state_in: the states before the first tokens or NULL
 * (zeros); state_out: receives the states after the last ones, or NULL; it may
 * be state_in.  o and state_out must not overlap other arrays (the same pointer is refused).  Bitwise
 * reproducible.  Sequences longer than some hundred tokens are cut into segments that run side by side
 * where few (sequence, head) pairs would leave the GPU idle, by a rule on n,
 * n_seq, heads and io_dtype alone: fewer than 128 pairs, and 8 times 64 tokens (fp32: 5
 * times) to a sequence on average.  The lengths themselves are on the device and
 * not looked at, so a long sequence among so many short ones that the rule leaves them
 * whole runs on one compute unit a head, 6 us to each 64 tokens: 100,000 tokens of 8
 * heads beside 16 sequences of 100 take 9.6 ms, alone or beside 14 of them 1.0. */
ZM_API int zm_delta_rule(const zm_delta_desc* desc, int64_t n, const int32_t* offsets,
                  const void* q, const void* k, const void* v, const float* g, const float* beta,
                  const float* state_in, float* state_out, void* o,
                  void* workspace, size_t workspace_bytes, void* stream);

/* One token of each of n_seq sequences (row b: sequence b), states updated in
 * place.  o must not overlap another array (the same pointer is refused).  No workspace. */
ZM_API int zm_delta_rule_step(const zm_delta_desc* desc, const void* q, const void* k, const void* v,
                       const float* g, const float* beta, float* state, void* o, void* stream);

/* Bytes of workspace of zm_delta_rule_backward for n tokens in desc->n_seq sequences (never
 * less for more tokens).  The states are formed again and kept chunk by chunk: to each 64
 * tokens (or begun 64 of a sequence) of a value head 3.6 states of 128 x 128, or 6.3 of
 * 64 x 64; 0.3 (1.2) more with fp32 tokens and 1 (2) more with shared key heads; and
 * where sequences are cut, 6 more to each of at most n_seq + 256 / heads segments of a head. */
ZM_API int zm_delta_rule_backward_workspace_size(const zm_delta_desc* desc, int64_t n, size_t* bytes);

/* The gradient of zm_delta_rule from its inputs alone: d_o [n, heads, d_head]
 * (stride desc->ld_o) and dstate_out (gradient of the last states, NULL: zeros)
 * give dq, dk [n, heads_k, d_head] (summed over the value heads of a key head),
 * dv [n, heads, d_head] in the io type, dg, dbeta fp32 [n, heads] and
 * dstate_in (NULL: not wanted).  Token strides as in the descriptor.  Rows
 * outside every sequence are left as they were.  The outputs must not overlap the inputs
 * or each other (the same pointer is refused; dstate_in may be dstate_out).  dg is a difference of
 * sums, good to some 2^-24 of the state times its gradient: where a strong decay makes it far
 * smaller than those, and below g = -128 (a reset), it is zero up to that rounding.  Bitwise reproducible. */
ZM_API int zm_delta_rule_backward(const zm_delta_desc* desc, int64_t n, const int32_t* offsets,
                  const void* d_o, const void* q, const void* k, const void* v, const float* g,
                  const float* beta, const float* state_in, const float* dstate_out,
                  void* dq, int64_t ld_dq, void* dk, int64_t ld_dk, void* dv, int64_t ld_dv,
                  float* dg, float* dbeta, float* dstate_in,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Linear attention with decays: the linear fast weight f_S(x) = S x written by adding
 * v_t k_t^T (the delta rule above without taking S k_t off), with a decay to each head:
 *   S_t = a_t S_{t-1} + v_t k_t^T,  a_t = exp(g_t),  o_t = scale S_t q_t.
 * Tokens, heads, offsets and states as for zm_delta_rule.  g (log decay; -inf resets the state)
 * is fp32, token t's of value head h at g[t ld_g + h]: ld_g >= heads, or ld_g = 0 for one decay
 * to each head, the same for every token; NULL: no decay, a = 1.  A decay may be above 0, but no run of a
 * sequence's tokens may have a sum of g over 40.
 * A token that is not finite can make NaN, in its heads, of the outputs of the 64 tokens
 * (fp32: 32) that it is taken with (counted from its sequence's first) and of later ones and of its
 * sequence's gradients; earlier chunks' outputs and other sequences stay as they are.
 * Products are held beside powers of two of up to 2^60.  So all of these stay below 2^60: values of tokens
 * and states (those on the way too), |q|.|k|, |S| |q|, and |k| |v| and (|q|.|k|) |v| added up over 64 tokens; in the gradient the same
 * with d_o and states' gradients in the places of others, and where dg is wanted also (|q|.|k|) (|d_o|.|v|),
 * (|S| |q|).|d_o| and <|S|, |dS|>, each times |scale| where that is over 1.  Tokens up to 2^10 and states up
 * to 2^20 in size do with a scale of at most 1. */
typedef struct zm_linear_desc {
  int32_t heads;      /* value heads, 1..64, a multiple of heads_k */
  int32_t heads_k;    /* query/key heads */
  int32_t d_head;     /* 64 or 128 */
  int32_t io_dtype;   /* zm_dtype of q, k, v, o and their gradients */
  int32_t n_seq;      /* sequences, >= 0 */
  float scale;        /* of the outputs */
  int64_t ld_q, ld_k, ld_v, ld_o;  /* token strides: >= heads * d_head (q, k: heads_k *
                                      d_head), multiples of 8, at most 2^24 */
  int64_t ld_g;       /* 0, or heads .. 2^24 */
} zm_linear_desc;

/* Bytes of workspace of zm_linear_attention for n tokens in desc->n_seq sequences (never less
 * for more tokens): at most 1024 / heads states to a head, and past 64 sequences a table of 32
 * bytes to a sequence. */
ZM_API int zm_linear_attention_workspace_size(const zm_linear_desc* desc, int64_t n, size_t* bytes);

/* Whole sequences, a chunk of tokens at a time (fp32 states; products of 24 bits up to the
 * rounding of an output).  state_in: the states before the first tokens or NULL (zeros);
 * state_out: receives the states after the last ones, or NULL; it may be state_in.
 * o and state_out must not overlap other arrays (the same pointer is refused).  Rows of o
 * outside every sequence are left as they were.  Bitwise reproducible.  A sequence is cut into
 * segments of a length that follows from n, n_seq, heads and io_dtype alone, which run side by
 * side. */
ZM_API int zm_linear_attention(const zm_linear_desc* desc, int64_t n, const int32_t* offsets,
                  const void* q, const void* k, const void* v, const float* g,
                  const float* state_in, float* state_out, void* o,
                  void* workspace, size_t workspace_bytes, void* stream);

/* One token of each of n_seq sequences (row b: sequence b), states updated in place.
 * o must not overlap another array (the same pointer is refused).  No workspace. */
ZM_API int zm_linear_attention_step(const zm_linear_desc* desc, const void* q, const void* k, const void* v,
                       const float* g, float* state, void* o, void* stream);

/* Bytes of workspace of zm_linear_attention_backward (never less for more tokens): the forward's
 * twice, with shared key heads two fp32 copies of the value heads' tokens, and for dg to each 64
 * tokens (fp32: 32; or begun ones of a sequence) of a value head a state.  The second: of calls
 * whose dg is NULL. */
ZM_API int zm_linear_attention_backward_workspace_size(const zm_linear_desc* desc, int64_t n, size_t* bytes);
ZM_API int zm_linear_attention_backward_workspace_size_no_dg(const zm_linear_desc* desc, int64_t n, size_t* bytes);

/* The gradient of zm_linear_attention from its inputs alone: d_o [n, heads, d_head] (stride
 * desc->ld_o) and dstate_out (gradient of the last states, NULL: zeros) give dq, dk [n, heads_k,
 * d_head] (summed over the value heads of a key head), dv [n, heads, d_head] in the io type, dg
 * (NULL: not wanted, as it has to be without g) and dstate_in (NULL: not wanted).  dg is fp32
 * [n, heads] contiguous, or, with ld_g = 0, [heads]: summed over all tokens.  Rows outside every
 * sequence are left as they were.  The outputs must not overlap the inputs or each other (the
 * same pointer is refused; dstate_in may be dstate_out).  dg_t is formed of terms that each hold
 * the factor a_t, so it is as good as fp32 products where decays are strong too; below
 * g = -128 it is zero.  Bitwise reproducible. */
ZM_API int zm_linear_attention_backward(const zm_linear_desc* desc, int64_t n, const int32_t* offsets,
                  const void* d_o, const void* q, const void* k, const void* v, const float* g,
                  const float* state_in, const float* dstate_out,
                  void* dq, int64_t ld_dq, void* dk, int64_t ld_dk, void* dv, int64_t ld_dv,
                  float* dg, float* dstate_in,
                  void* workspace, size_t workspace_bytes, void* stream);

/* Gradients' global norm and clipping: N = sqrt(sum of x^2 over all elements of all
 * tensors), y = x min(1, max_norm / (N + 1e-6)).  Sums are in 64 bits, where N is finite for finite
 * elements: past fp32's range norm receives infinity, and y is formed with N all the same.  Infinite
 * elements make y 0 (NaN where x is infinite), NaN ones make every y NaN. */
typedef struct zm_tensor {
  const void* x;      /* n elements one after the other, aligned to one */
  void* y;            /* where the clipped ones go: x itself, or an array of its own */
  int64_t n;          /* 0..2^36; of none the pointers are not looked at */
  int32_t dtype;      /* zm_dtype of x and y */
  int32_t reserved;   /* must be 0 */
} zm_tensor;

/* Bytes of workspace of the two calls below for `count` tensors (at most 8192). */
ZM_API int zm_grad_norm_workspace_size(int32_t count, size_t* bytes);

/* norm (device, fp32): N.  tensors is host memory that is read during the call alone; the ys
 * are not looked at.  The workspace must not overlap a tensor; tensors may overlap each
 * other.  Bitwise reproducible, as the next. */
ZM_API int zm_grad_norm(const zm_tensor* tensors, int32_t count, float* norm,
              void* workspace, size_t workspace_bytes, void* stream);

/* Writes every y, and N (before clipping) to norm.  max_norm: finite, >= 0.  No array may
 * overlap another one (x may be its own y). */
ZM_API int zm_clip_grads(const zm_tensor* tensors, int32_t count, float max_norm, float* norm,
              void* workspace, size_t workspace_bytes, void* stream);

/* Static description of a status code. */
ZM_API const char* zm_status_string(int status);

/* The slow weights around the layer: the projections of an input token x
 * (width d_in) to q, k, v (ZipMap notes, q / k / v 投影) and to the per-token
 * rate (review, note under Eq. (3): a linear layer of the token), and the
 * output gate of review Eq. (5).  Readings where the pages are silent: the
 * rate is eta = eta_scale * sigmoid(W_eta x); RMSNorm runs over the whole
 * width H * d_head with a learnable scale gamma and epsilon rms_eps. */
typedef struct zm_layer_weights {
  const void* w_in;     /* bf16 [3 H d + H][d_in]: rows of W_Q, W_K, W_V (H d each,
                           head-major, d_head consecutive rows per head), then W_eta (H) */
  const void* w_gate;   /* bf16 [H d][H d]: W_g */
  const float* gamma;   /* fp32 [H d]: RMSNorm scale, 16-byte aligned */
  int32_t d_in;         /* input width, a multiple of 8 */
  float eta_scale;      /* >= 0 */
  float rms_eps;        /* > 0 */
  int32_t reserved;     /* must be 0 */
} zm_layer_weights;

/* Bytes of workspace zm_ttt_layer needs for n tokens. */
ZM_API int zm_ttt_layer_workspace_size(const zm_ttt_desc* desc, const zm_layer_weights* lw,
                                int64_t n, size_t* bytes);

/* The whole TTT layer on one bidirectional chunk of n tokens x (bf16 rows of
 * stride ld_x, ld_x >= d_in, a multiple of 8):
 *   [q | k | v | z] = W_in x,  eta = eta_scale * sigmoid(z),
 *   W_hat = update(W; k, v, eta) (+ renorm, desc->step_rule),
 *   o' = f_{W_hat}(q),  o = RMSNorm(o') * SiLU(W_g o')  (review Eq. (5)).
 * desc: heads, d_head, d_hidden, renorm and step_rule as for the other entry
 * points, with a layer width H d of at most 8192 (wider: ZM_ERR_UNSUPPORTED);
 * io_dtype must be ZM_BF16; desc->ld_tok is the row stride of o
 * (>= H d, a multiple of 8).  w1..w3 are read, W_hat goes to w*_out (may
 * alias).  o: bf16 [n][H d].  The projections and W_g o' run as library GEMMs
 * (bf16 operands, fp32 accumulation, bf16 results); the rate, the gate and the
 * TTT steps run in the library's kernels. */
ZM_API int zm_ttt_layer(const zm_ttt_desc* desc, const zm_layer_weights* lw, int64_t n,
                 const void* x, int64_t ld_x, const float* w1, const float* w2, const float* w3,
                 float* w1_out, float* w2_out, float* w3_out, void* o,
                 void* workspace, size_t workspace_bytes, void* stream);

/* Description of the last ZM_ERR_HIP failure on the calling thread (the HIP
 * call or GEMM-library call that failed and its status), or "" if none.
 * The string stays valid until the thread's next failing call. */
ZM_API const char* zm_ttt_last_error(void);

/* Library version as major*10000 + minor*100 + patch.  Entry points that came
 * beside the others, none of which changed (zm_layer_norm, zm_rotary, zm_delta_rule, zm_linear_attention,
 * zm_norm_rotary, zm_grad_norm, zm_clip_grads and theirs),
 * left the number as it was: a program that loads the library at run time looks for
 * their symbols. */
ZM_API int zm_ttt_version(void);

/* Profiling aid: when events != NULL, every later launch of kernel stage s
 * (0 weight cast, 1 update partial sums, 2 reduce/step/renorm, 3 apply,
 * 4 Newton-Schulz, 5 input projections and rate, 6 output gate) records
 * events[2s] before and events[2s+1] after itself on the launch stream, for
 * each non-NULL slot.  Where a chunk's read and its update's partial sums
 * share one launch (bf16 APPLY_THEN_UPDATE), the events of stages 1 and 3
 * both bracket that launch; where the reduce runs inside the update's launch
 * (short chunks, see Workspace above), so do those of stage 2.  The events are hipEvent_t handles passed as void*;
 * n_events must be 8 (stages 0-3), 10 (0-4) or 14 (0-6) (or 0 with
 * events == NULL to switch off).  Process-wide setting; not for concurrent use
 * from several threads. */
ZM_API int zm_ttt_set_profile_events(void* const* events, int n_events);

#ifdef __cplusplus
}
#endif

#endif /* ZM_TTT_H */
