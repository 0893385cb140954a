/*
 * kda.h -- C ABI of the MI355X (gfx950) Kimi Delta Attention library, libkda.so.
 *
 * The layer (one head, state S with dk rows = key channels and dv columns):
 * for every token t, in order,
 *     S <- Diag(exp(g_t)) S                       fade each key channel
 *     S <- S + beta_t k_t (v_t - S^T k_t)^T       erase what k_t retrieves, write v_t
 *     o_t = S^T q_t                               read from the updated state
 * ("Review A - Sequence and depth", Free recall, the question on KDA's three
 * operations; "K3 Architecture Illustrated", section "Combining KDA and MLA",
 * FIG 21; the erase factor I - beta k k^T from the section "Under what
 * conditions are RoPE, PaTH, and KDA related?").
 *
 * kda_chunk_fwd computes this over a whole sequence in the chunkwise form:
 * sequential between 64-token chunks, parallel inside a chunk, with the
 * output split into the inter-chunk term (Gamma . Q) S and the masked
 * intra-chunk term A V~, and keys rescaled by 1/Gamma inside 16-token tiles
 * ("Kimi K3 - Lesson 3 of 14 - Sequence axis", the chunkwise diagram and the
 * paragraphs on the 1/Gamma rescale and on g_min = -5).  The result is the
 * token recurrence's, up to rounding.
 *
 * kda_decode_step advances every (sequence, head) state by one token in place
 * (the fixed-size state of "Review A", Discriminating between mechanisms).
 *
 * kda_verify_step and kda_commit_step serve speculative decoding ("K3
 * Architecture Illustrated", the section on speculative decoding: the
 * recurrent state needs rollback handling after rejected proposals): verify
 * runs K draft tokens through the current state without changing it, commit
 * then advances the state by each sequence's accepted prefix only.
 *
 * kda_chunk_fwd_gate and kda_decode_step_gate take raw gate logits z and a
 * per-head log-scale A_h instead of g, and form g = -5 sigmoid(exp(A_h) z)
 * inside the kernels ("Kimi K3 - Lesson 3 of 14 - Sequence axis", the
 * scaled-sigmoid gate with g_min = -5 and A_h a learnable per-head log-scale
 * initialised to 0).  The page shows the mapping without its formula; the
 * scale is read as acting on the logit inside the sigmoid, which keeps every
 * g in [-5, 0] for any A_h and is the plain -5 sigmoid(z) at A_h = 0.
 *
 * kda_output_gate and kda_decode_step_gated apply the module's output
 * epilogue to the read: per (token, head) row of dv channels
 *     y = o / sqrt(mean_j o_j^2 + eps) * weight * sigmoid(z_out)
 * ("Kimi K3 - Lesson 3 of 14 - Sequence axis", the output-gate paragraph: a
 * full-rank, input-dependent gate after the recurrent read decides which
 * channels pass; "K3 Architecture Illustrated", the KDA section under FIG 21:
 * the module includes normalisation and output gating).  The pages give no
 * formula; the reading is RMS normalisation over the head's dv channels with
 * a learnable per-channel weight [dv] shared by all heads, then a sigmoid
 * gate from per-token logits with o's shape.
 *
 * Conventions for every entry point
 * ---------------------------------
 *  - Tensor pointers are DEVICE pointers to contiguous row-major memory, each
 *    aligned to 16 bytes.  The caller owns every buffer; the library
 *    allocates nothing, keeps no state between calls and is reentrant.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Work is enqueued
 *    asynchronously on it; device-side faults surface at the caller's next
 *    synchronisation.
 *  - Arguments are validated on the host before any HIP call.  A non-OK
 *    status means nothing was enqueued (KDA_ERR_LAUNCH: the launch itself
 *    was rejected by the runtime).
 *  - Preconditions that are NOT checked (the data stays on the device):
 *    every g lies in [-5, 0] (the g_min = -5 floor that bounds 1/Gamma by e^80
 *    inside a 16-token tile, "Kimi K3 - Lesson 3 of 14", the g_min
 *    paragraphs); all inputs are finite.  Outside them results are undefined
 *    (typically inf/NaN), never a fault.
 *  - Keys and queries are used as given (no normalisation, no scaling).
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Both enums span the whole int range (the two range members), so any int a
 * caller passes is a value of the type: out-of-set values are rejected by
 * the checks, not undefined behaviour. */
typedef enum {
    KDA_F32 = 0,   /* IEEE float32 */
    KDA_BF16 = 1,  /* bfloat16 (round-to-nearest-even when produced) */
    KDA_DTYPE_RANGE_MIN_ = -2147483647 - 1,
    KDA_DTYPE_RANGE_MAX_ = 2147483647
} kda_dtype_t;

/* The cache's 8-bit codes: a value is its code times the scale of its page and head. */
typedef enum {
    KDA_CODE_E4M3 = 0, /* 8-bit float: 4 exponent and 3 mantissa bits, largest 448, no infinities */
    KDA_CODE_INT8 = 1, /* integer, -127 .. 127 */
    KDA_CODE_RANGE_MIN_ = -2147483647 - 1,
    KDA_CODE_RANGE_MAX_ = 2147483647
} kda_code_t;

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,  /* NULL / misaligned / overlapping pointer, negative size, bad dtype */
    KDA_ERR_UNSUPPORTED = 2,  /* valid but not provided: dk or dv outside the supported set */
    KDA_ERR_LAUNCH = 3,       /* the HIP runtime rejected the kernel launch */
    KDA_ERR_SCRATCH = 4,      /* kda_chunk_fwd_noalloc: input beyond its fixed scratch */
    KDA_STATUS_RANGE_MIN_ = -2147483647 - 1,
    KDA_STATUS_RANGE_MAX_ = 2147483647
} kda_status_t;

/* ABI version of this header; bumped on any incompatible change. */
#define KDA_ABI_VERSION 6

/*
 * kda_chunk_fwd -- chunkwise forward over T tokens for B sequences x H heads.
 *
 *   q, k   [B, T, H, dk]  qkv_dtype   queries, keys
 *   v      [B, T, H, dv]  qkv_dtype   values
 *   g      [B, T, H, dk]  gate_dtype  per-key-channel log-decay, in [-5, 0]
 *   beta   [B, T, H]      gate_dtype  write strength (any real value)
 *   S0     [B, H, dk, dv] float32     initial state, or NULL for zeros
 *   o      [B, T, H, dv]  out_dtype   output (written)
 *   S_final[B, H, dk, dv] float32     state after token T-1 (written), or NULL
 *                                     to skip; may be the same pointer as S0
 *                                     (in-place continuation), must not
 *                                     overlap it otherwise.
 *
 * Supported: dk in {64, 128}; dv a positive multiple of 64, at most 512;
 * any T >= 0 (a ragged final chunk is padded internally with identity
 * tokens, which leave the state unchanged); B, H >= 0.  T == 0 copies S0
 * (or zeros) to S_final.  `o` must not overlap any input; S_final must not
 * overlap q, k, v, g, beta or o.
 *
 * Internal state is float32.  Contractions run on the matrix cores with
 * float32 accumulation: float32 operands when qkv_dtype == KDA_F32; for
 * KDA_BF16 inputs, fp16 operands (11 significant bits), with the state-update
 * operand U and the right-hand sides of the diagonal solves carried as two
 * fp16 terms, and two-term bfloat16 for the diagonal 16-token Gram tiles,
 * whose 1/decay factor reaches e^80.  The fp16 operands need |v|, |S| and
 * |o| below 65504 (true for unit-scale values and L2-normalised q and k, as
 * the method uses them); beyond that the KDA_BF16 path produces inf.
 * out_dtype == KDA_F32 keeps the output at accumulator precision; KDA_BF16
 * rounds it once (the output of a heavy-tailed workload can lose several
 * percent of its RMS to that rounding alone).
 */
kda_status_t kda_chunk_fwd(const void *q, const void *k, const void *v,
                           const void *g, const void *beta, const float *S0,
                           void *o, float *S_final,
                           int B, int T, int H, int dk, int dv,
                           kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype,
                           kda_dtype_t out_dtype, void *stream);

/*
 * kda_decode_step -- one token for every (sequence, head), state updated in place.
 *
 *   q, k   [B, H, dk]     qkv_dtype
 *   v      [B, H, dv]     qkv_dtype
 *   g      [B, H, dk]     gate_dtype  log-decay in [-5, 0]
 *   beta   [B, H]         gate_dtype
 *   S      [B, H, dk, dv] float32     read and written IN PLACE
 *   o      [B, H, dv]     out_dtype   output (written)
 *
 * Supported: dk in {64, 128}, dv in {64, 128}; B, H >= 0.  `o` must not
 * overlap any input or S; S must not overlap q, k, v, g or beta.
 * Arithmetic is float32 throughout (the step is bandwidth-bound).
 */
kda_status_t kda_decode_step(const void *q, const void *k, const void *v,
                             const void *g, const void *beta, float *S, void *o,
                             int B, int H, int dk, int dv,
                             kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype,
                             kda_dtype_t out_dtype, void *stream);

/*
 * kda_chunk_fwd_gate -- kda_chunk_fwd with the log-decay formed in the kernel.
 *
 *   z      [B, T, H, dk]  gate_dtype  gate logits (any real value)
 *   A_log  [H]            float32     per-head log-scale A_h (device pointer,
 *                                     4-byte aligned)
 *   g = -5 sigmoid(exp(A_log[h]) z), in [-5, 0] for every z.  Everything
 *   else, including supported sizes and errors, as kda_chunk_fwd; A_log must
 *   not be NULL and must not overlap o or S_final.
 */
kda_status_t kda_chunk_fwd_gate(const void *q, const void *k, const void *v,
                                const void *z, const float *A_log, const void *beta,
                                const float *S0, void *o, float *S_final,
                                int B, int T, int H, int dk, int dv,
                                kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype,
                                kda_dtype_t out_dtype, void *stream);

/*
 * kda_chunk_fwd_ws, kda_chunk_fwd_gate_ws -- kda_chunk_fwd and
 * kda_chunk_fwd_gate with a caller-owned workspace.  The workspace lets
 * bfloat16 q, k, v with dk = 128 (dv a multiple of 64 from 128 to 512) take
 * the ring kernel: a head's dv columns are split over dv / 64 workgroups,
 * which take turns computing the state-independent part of the chunks of the
 * chunkwise form ("Kimi K3 - Lesson 3 of 14 - Sequence axis", the chunkwise
 * diagram: decays, 1/Gamma-rescaled operands, intra-chunk Gram tiles, the
 * diagonal inverses), so each chunk's part is computed once per head instead
 * of once per workgroup, and hand it to one another through a four-slot ring
 * per head held in the workspace.  Other inputs run the kernels of
 * kda_chunk_fwd.  The ring pays for dv of 256 and more when the grid (B H dv
 * / 64 workgroups) fills at most half the device (at B = 1, H = 8, T = 4096:
 * 1.0x the time of kda_chunk_fwd at dv = 128, 0.84x at dv = 256, 0.79x at
 * dv = 512); a full-device grid runs faster without it (1.28x at B = 1, H =
 * 96, T = 131072, dv = 128).
 *
 *   workspace        device memory of at least kda_chunk_fwd_workspace_bytes(B,
 *                    T, H, dk, dv) bytes, 16-byte aligned, owned by the caller;
 *                    it needs no initialisation, its contents are undefined
 *                    afterwards, and it must not overlap any other argument.
 *                    NULL makes the call kda_chunk_fwd (or _gate) exactly.
 *   workspace_bytes  its size; a non-NULL workspace below the required size is
 *                    KDA_ERR_INVALID_ARG.
 *
 * Everything else (shapes, dtypes, aliasing rules, preconditions, precision,
 * errors) as kda_chunk_fwd / kda_chunk_fwd_gate; the arithmetic is the same,
 * step for step.  Calls sharing one workspace must not overlap in time (use
 * one stream, or one workspace per stream).  The kernel's workgroups wait
 * for one another (bounded waits, at most kda_debug_set_spin_limit sleeps
 * each); if a wait runs out, the call still completes and every output it
 * writes from then on (o and S_final of the affected heads) is NaN.
 */
size_t kda_chunk_fwd_workspace_bytes(int B, int T, int H, int dk, int dv);   /* 0: no workspace is used */

kda_status_t kda_chunk_fwd_ws(const void *q, const void *k, const void *v,
                              const void *g, const void *beta, const float *S0,
                              void *o, float *S_final, void *workspace, size_t workspace_bytes,
                              int B, int T, int H, int dk, int dv,
                              kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype,
                              kda_dtype_t out_dtype, void *stream);

kda_status_t kda_chunk_fwd_gate_ws(const void *q, const void *k, const void *v,
                                   const void *z, const float *A_log, const void *beta,
                                   const float *S0, void *o, float *S_final,
                                   void *workspace, size_t workspace_bytes,
                                   int B, int T, int H, int dk, int dv,
                                   kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype,
                                   kda_dtype_t out_dtype, void *stream);

/*
 * kda_chunk_fwd_noalloc -- kda_chunk_fwd_ws for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc): the ring lives in a device array inside the library
 * instead of a caller's workspace.  The call allocates nothing and calls no
 * allocating routine.
 *
 * Arguments, preconditions, results and errors as kda_chunk_fwd_ws without
 * the workspace.  The array holds the ring of 64 heads (about 15.8 MiB per
 * device, kept until the process ends): where the ring kernel applies
 * (bfloat16 q, k, v, dk = 128, dv a multiple of 64 from 128 to 512) and B * H
 * exceeds 64, the call returns KDA_ERR_SCRATCH and enqueues nothing; other
 * inputs run the kernels of kda_chunk_fwd, which use no scratch.  Every call
 * on one device shares that device's array: calls that overlap in time on one
 * device (two streams, two threads) race and give undefined results; calls
 * ordered on one stream do not.  The array's contents carry over from call to
 * call and need no clearing (each launch tags its flags with a fresh epoch).
 */
kda_status_t kda_chunk_fwd_noalloc(const void *q, const void *k, const void *v,
                                   const void *g, const void *beta, const float *S0,
                                   void *o, float *S_final, int B, int T, int H, int dk, int dv,
                                   kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype,
                                   kda_dtype_t out_dtype, void *stream);

/*
 * kda_chunk_fwd_seqpar -- kda_chunk_fwd computed as `segments` pieces of the
 * sequence side by side, for grids too small to fill the device (few
 * sequences and heads, long T).  Between chunks the chunkwise form is a
 * sequential recurrence ("Kimi K3 - Lesson 3 of 14 - Sequence axis", the
 * chunkwise diagram), but each chunk's step is affine in the state, so a run
 * of chunks is too: S_out = M S_in + N.  The call runs every segment of
 * T / segments tokens from a zero state, also carrying dk transition columns
 * that start from the identity with zero values (giving N and M per segment),
 * forms the segments' true starting states in order (S_{p+1} = M_p S_p + N_p
 * in float32; the last one is S_final), and runs every segment again from its
 * starting state to write o.  The sequential part is T / segments tokens long
 * twice instead of T once, at (dv + dk) / dv times the first pass's columns.
 * Results equal kda_chunk_fwd's up to rounding (the chunks start at every
 * segment start, and the segments meet through the float32 products).
 *
 *   segments   1 .. KDA_SEQPAR_MAX_SEGMENTS, dividing T; it pays while
 *              B * segments * H * (dv + dk) / 64 workgroups fit the device.
 *   workspace  device memory of at least kda_chunk_fwd_seqpar_workspace_bytes
 *              bytes, 16-byte aligned, owned by the caller, not overlapping any
 *              other argument; no initialisation needed, contents undefined
 *              afterwards.  Calls sharing one workspace must not overlap in time.
 *
 * Everything else (shapes, dtypes, S0 / S_final aliasing, preconditions,
 * precision, errors) as kda_chunk_fwd, with these additions: q, k, v must be
 * bfloat16 (KDA_ERR_UNSUPPORTED otherwise); segments outside the range or not
 * dividing T, or a missing or short workspace, is KDA_ERR_INVALID_ARG.
 */
#define KDA_SEQPAR_MAX_SEGMENTS 64
size_t kda_chunk_fwd_seqpar_workspace_bytes(int B, int T, int H, int dk, int dv, int segments);   /* 0: invalid shape */

/*
 * kda_chunk_fwd_seqpar_segments -- a segment count for kda_chunk_fwd_seqpar,
 * or 1 where the plain kda_chunk_fwd is expected to be faster.  Host-only
 * arithmetic on the shape: among the divisors of T up to
 * KDA_SEQPAR_MAX_SEGMENTS, the one with the smallest estimated time (passes
 * of B * segments * H * (dv + dk) / 64 and B * segments * H * dv / 64
 * workgroups over `cus` compute units, and the combine), compared with the
 * plain forward's, from per-chunk and per-segment costs measured on MI355X.
 * cus <= 0 takes the current device's compute-unit count (1 is returned if
 * that query fails).  Invalid shapes return 1.
 */
int kda_chunk_fwd_seqpar_segments(int B, int T, int H, int dk, int dv, int cus);

kda_status_t kda_chunk_fwd_seqpar(const void *q, const void *k, const void *v,
                                  const void *g, const void *beta, const float *S0,
                                  void *o, float *S_final, void *workspace, size_t workspace_bytes,
                                  int B, int T, int H, int dk, int dv, int segments,
                                  kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype,
                                  kda_dtype_t out_dtype, void *stream);

/*
 * kda_chunk_fwd_gate_seqpar -- kda_chunk_fwd_seqpar with the log-decay formed
 * in the kernels from gate logits z and per-head A_log, as kda_chunk_fwd_gate
 * does ("Kimi K3 - Lesson 3 of 14 - Sequence axis", the scaled-sigmoid
 * mapping).  Arguments as kda_chunk_fwd_seqpar with z in place of g and A_log
 * ([H] float32, device) added; a NULL A_log is KDA_ERR_INVALID_ARG.  The
 * workspace size is kda_chunk_fwd_seqpar_workspace_bytes'.
 */
kda_status_t kda_chunk_fwd_gate_seqpar(const void *q, const void *k, const void *v,
                                       const void *z, const float *A_log, const void *beta,
                                       const float *S0, void *o, float *S_final,
                                       void *workspace, size_t workspace_bytes,
                                       int B, int T, int H, int dk, int dv, int segments,
                                       kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype,
                                       kda_dtype_t out_dtype, void *stream);

/*
 * kda_debug_set_spin_limit -- test hook: the bound (sleeps between polls) on
 * every wait inside the chunk kernels launched after the call, process-wide;
 * returns the previous bound (default 2^20).  A small bound makes the waits
 * give up, which lets a test check that a failed wait yields NaN outputs
 * rather than wrong finite ones.  Not for production use.
 */
unsigned kda_debug_set_spin_limit(unsigned limit);

/*
 * kda_decode_step_gate -- kda_decode_step with g = -5 sigmoid(exp(A_log[h]) z)
 * formed in the kernel (z [B, H, dk] gate_dtype, A_log [H] float32).
 */
kda_status_t kda_decode_step_gate(const void *q, const void *k, const void *v,
                                  const void *z, const float *A_log, const void *beta,
                                  float *S, void *o, int B, int H, int dk, int dv,
                                  kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype,
                                  kda_dtype_t out_dtype, void *stream);

/*
 * kda_verify_step -- K draft tokens per sequence through the current state,
 * outputs only.
 *
 *   q, k, g [B, K, H, dk], v [B, K, H, dv], beta [B, K, H]: the draft tokens
 *   S       [B, H, dk, dv] float32   the state before the drafts; READ ONLY
 *   o       [B, K, H, dv]  out_dtype o[:, j] is the output token j would get
 *                                    after tokens 0..j-1 of its draft
 *
 * Equivalent to kda_chunk_fwd(q, k, v, g, beta, S0 = S, o, S_final = NULL)
 * over T = K tokens; same sizes, dtypes and errors.  S must not be NULL and
 * must not overlap o.  Up to 16 drafts run as one tile of the chunkwise form
 * on the matrix cores; with KDA_BF16 drafts its two products with the state
 * take single fp16 operands (so |S| must stay below 65504, as for
 * kda_chunk_fwd), with KDA_F32 drafts float32 operands.
 */
kda_status_t kda_verify_step(const void *q, const void *k, const void *v,
                             const void *g, const void *beta, const float *S, void *o,
                             int B, int K, int H, int dk, int dv,
                             kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype,
                             kda_dtype_t out_dtype, void *stream);

/*
 * kda_commit_step -- advance S in place by the accepted prefix of each draft.
 *
 *   k, g [B, K, H, dk], v [B, K, H, dv], beta [B, K, H]: the same draft tokens
 *   accepted [B] int32 (device): tokens 0..accepted[b]-1 of sequence b are
 *                   applied, the rest are treated as identity tokens (values
 *                   are clamped to [0, K])
 *   S        [B, H, dk, dv] float32, read and written IN PLACE
 *
 * Afterwards S is the state kda_chunk_fwd would reach over the first
 * accepted[b] tokens of each sequence.  No output is written.  S must not
 * overlap k, v, g, beta or accepted.  A sequence with no accepted token
 * keeps its state bit for bit.  Up to 16 drafts run as one tile on the
 * matrix cores (S read once, updated in registers, written once; of the
 * drafts only the accepted prefix is read from memory); with
 * KDA_BF16 drafts the products take two-term fp16 operands (about 22
 * significant bits; |S| below 65504), with KDA_F32 drafts float32 operands.
 */
kda_status_t kda_commit_step(const void *k, const void *v, const void *g, const void *beta,
                             const int *accepted, float *S,
                             int B, int K, int H, int dk, int dv,
                             kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype, void *stream);

/*
 * kda_output_gate -- the output epilogue over `rows` rows of dv channels
 * (rows = B * T * H for a forward's o [B, T, H, dv]).
 *
 *   o      [rows, dv] o_dtype       the reads
 *   z      [rows, dv] z_dtype       gate logits
 *   weight [dv] float32             per-channel normalisation weight
 *   eps    >= 0, finite             added to the mean square (eps = 0 makes an
 *                                   all-zero row NaN, as the formula does)
 *   y      [rows, dv] y_dtype       the result; may be o itself when
 *                                   y_dtype == o_dtype, must not overlap z or
 *                                   weight otherwise
 *
 * dv a multiple of 64 up to 512 (else KDA_ERR_UNSUPPORTED).  float32 arithmetic.
 */
kda_status_t kda_output_gate(const void *o, const void *z, const float *weight, float eps, void *y,
                             int64_t rows, int dv, kda_dtype_t o_dtype, kda_dtype_t z_dtype,
                             kda_dtype_t y_dtype, void *stream);

/*
 * kda_decode_step_gated -- a decode step whose output goes through the output
 * epilogue inside the same kernel: y = kda_output_gate(o) with o the read
 * kda_decode_step would write.
 *
 *   g       [B, H, dk] gate_dtype: the log-decay when A_log is NULL, gate
 *           logits (as kda_decode_step_gate) when A_log [H] float32 is given
 *   z_out   [B, H, dv] qkv_dtype    output-gate logits
 *   weight  [dv] float32, eps >= 0  as kda_output_gate
 *   y       [B, H, dv] out_dtype    the gated output (o itself is not stored)
 *
 * Otherwise as kda_decode_step; y must not overlap any input or S.
 */
kda_status_t kda_decode_step_gated(const void *q, const void *k, const void *v, const void *g,
                                   const float *A_log, const void *beta, float *S, const void *z_out,
                                   const float *weight, float eps, void *y, int B, int H, int dk, int dv,
                                   kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype, kda_dtype_t out_dtype,
                                   void *stream);

/*
 * kda_chunk_bwd -- gradients of kda_chunk_fwd.  Given the upstream gradients
 * dO of the outputs (and dS_final of the final state), computes the
 * gradients of L = sum(o * dO) + sum(S_final * dS_final) with respect to
 * q, k, v, g, beta and S0.  The pages describe training the layer but give
 * no gradients; these are the derivatives of the recurrence above, taken
 * through the chunkwise form (32-token chunks, tile-local 1/Gamma references
 * as in the forward, float32 arithmetic throughout).
 *
 *   q, k, v, g, beta, S0   as kda_chunk_fwd (S0 NULL = zero state)
 *   dO        [B, T, H, dv]  do_dtype
 *   dS_final  [B, H, dk, dv] float32, or NULL (= zero)
 *   dq, dk, dg [B, T, H, dk], dv [B, T, H, dv], dbeta [B, T, H]: float32 outputs
 *   dS0       [B, H, dk, dv] float32 output, or NULL (not written)
 *   workspace device memory of at least kda_chunk_bwd_workspace_bytes(B, T,
 *             H, dk, dv) bytes, owned by the caller, contents undefined
 *             before and after; it must not overlap any argument
 *
 * dk, dv in {64, 128} (else KDA_ERR_UNSUPPORTED).  No output may overlap an
 * input, another output or the workspace.  Preconditions as the forward.
 */
size_t kda_chunk_bwd_workspace_bytes(int B, int T, int H, int dk, int dv);

kda_status_t kda_chunk_bwd(const void *q, const void *k, const void *v, const void *g, const void *beta,
                           const float *S0, const void *dO, const float *dS_final,
                           float *dq, float *dk, float *dv, float *dg, float *dbeta, float *dS0,
                           void *workspace, size_t workspace_bytes,
                           int B, int T, int H, int dk_dim, int dv_dim,
                           kda_dtype_t qkv_dtype, kda_dtype_t gate_dtype, kda_dtype_t do_dtype,
                           void *stream);

/*
 * Short causal convolution, selective state space scan and layer norm: the
 * rest of a recurrent block around the layer above.  Common to these calls:
 *
 *  - One storage type per call (`dtype`: KDA_F32 or KDA_BF16) for every
 *    per-token tensor, inputs, outputs and their gradients alike; parameters,
 *    states of the scan and parameters' gradients are float32.  Arithmetic,
 *    sums and states are float32; each output is rounded once, when stored.
 *  - D (channels) and T are any size >= 0; a call with nothing to compute
 *    still writes what its contract defines (states copied, gradients zero).
 *    Without channels (D = 0) a call returns at once and writes nothing; that
 *    leaves dBm and dCm of the scan's gradients, zeros by the formula, to the
 *    caller (the Python binding fills them).
 *    B T D, and every tensor's element count, must stay below 2^40, B, T and
 *    D below 2^24 each (KDA_ERR_UNSUPPORTED beyond).  So is a call whose grid
 *    would reach HIP's limit of 2^32 threads, before anything is enqueued: a
 *    convolution has one thread per sequence, run of 4 to 256 tokens and 1 to
 *    8 channels, a scan 256 per sequence, group, 64 channels and segment, its
 *    gradients 2 per sequence, channel and 16, 32 or 64 states besides.
 *  - lengths [B] int32 (device, or NULL: all T) are the sequences' lengths in
 *    a right-padded batch, clamped to [0, T].  Tokens behind a sequence's end
 *    enter no result (they may hold anything, NaN included); their outputs and
 *    their gradients are written as zeros, and final states are those after
 *    the last real token.
 *  - A workspace is device memory owned by the caller, 16-byte aligned, of at
 *    least the bytes the call's _workspace_bytes function gives (0: none
 *    needed, NULL allowed); no initialisation needed, contents undefined
 *    afterwards.  Calls sharing one workspace must not overlap in time.
 *  - No output may overlap an input, another output or the workspace, except
 *    where stated.  Results do not depend on timing: no atomics are used.
 */

/*
 * kda_short_conv_fwd -- depthwise causal convolution over the last W tokens of
 * each channel, with an optional SiLU.
 *
 *   pre[b, t, d] = bias[d] + sum_{j < W} w[d, j] x[b, t - W + 1 + j, d]
 *   y = pre * sigmoid(pre) if silu != 0, else pre
 *
 *   x            [B, T, D]      dtype
 *   w            [D, W] float32 (tap W - 1 is the current token's), bias [D] float32 or NULL
 *   state0       [B, W - 1, D]  dtype: the W - 1 inputs in front of token 0, oldest first;
 *                               NULL for zeros
 *   y            [B, T, D]      dtype (written)
 *   state_final  [B, W - 1, D]  dtype: the last W - 1 inputs (of state0 followed by the
 *                               sequence), written unless NULL; may be state0 itself
 *
 * W in {2, 3, 4} (KDA_ERR_UNSUPPORTED otherwise).
 */
kda_status_t kda_short_conv_fwd(const void *x, const float *w, const float *bias, const void *state0,
                                const int *lengths, void *y, void *state_final,
                                int B, int T, int D, int W, int silu, kda_dtype_t dtype, void *stream);

/*
 * kda_short_conv_step -- one token per sequence: x [B, D], y [B, D], and
 * state [B, W - 1, D] shifted by one token IN PLACE.  y may be x itself.
 */
kda_status_t kda_short_conv_step(const void *x, const float *w, const float *bias, void *state, void *y,
                                 int B, int D, int W, int silu, kda_dtype_t dtype, void *stream);

/*
 * kda_short_conv_bwd -- gradients of kda_short_conv_fwd for the upstream
 * gradients dy [B, T, D] of y and dstate_final [B, W - 1, D] (dtype, or NULL)
 * of state_final.
 *
 *   dx [B, T, D] dtype, dw [D, W] float32, dbias [D] float32 or NULL,
 *   dstate0 [B, W - 1, D] dtype or NULL (written unless NULL)
 */
size_t kda_short_conv_bwd_workspace_bytes(int B, int T, int D, int W);

kda_status_t kda_short_conv_bwd(const void *dy, const void *x, const float *w, const float *bias,
                                const void *state0, const void *dstate_final, const int *lengths,
                                void *dx, float *dw, float *dbias, void *dstate0,
                                void *workspace, size_t workspace_bytes,
                                int B, int T, int D, int W, int silu, kda_dtype_t dtype, void *stream);

/*
 * kda_selective_scan_fwd -- the selective state space recurrence: every
 * channel d carries N states that fade at rates A[d, :] times the token's own
 * time step, and takes its input through the token's own B and C rows.
 *
 *   s = dt + dt_bias, or softplus(dt + dt_bias) if softplus != 0
 *   h[d, n] <- exp(s[d] A[d, n]) h[d, n] + s[d] x[d] Bm[g, n],   g = d / (D / G)
 *   y[d] = (sum_n Cm[g, n] h[d, n] + Dskip[d] x[d]) * (z[d] sigmoid(z[d]))
 *
 *   x, dt    [B, T, D]     dtype
 *   A        [D, N] float32; A <= 0 keeps the states bounded (not checked).  Rates below
 *            -2.3586e38, -infinity among them, count as that one, which forgets at
 *            every positive step.  Where a segment's decay overflows (A > 0) or
 *            underflows in front of an infinite state, the state may be NaN earlier
 *            than token by token
 *   Bm, Cm   [B, T, G, N]  dtype; G groups of D / G channels each share them
 *   Dskip    [D] float32 or NULL (0);  dt_bias [D] float32 or NULL (0)
 *   z        [B, T, D]     dtype, or NULL: no gate
 *   h0       [B, D, N] float32, or NULL for zeros
 *   y        [B, T, D]     dtype (written)
 *   h_final  [B, D, N] float32 (written), or NULL; may be h0 itself
 *   workspace: with at least kda_selective_scan_fwd_workspace_bytes bytes the
 *            sequence is cut into segments run side by side and joined through
 *            their decays and end states; NULL runs each channel's tokens in one
 *            chain (the same results up to float32 rounding, slower where B D
 *            does not fill the device)
 *
 * N from 1 to 64, G >= 1 dividing D (KDA_ERR_INVALID_ARG if it does not);
 * the states take the room of 16, 32 or 64.  G N below 2^24.
 */
size_t kda_selective_scan_fwd_workspace_bytes(int B, int T, int D, int N, int G);

kda_status_t kda_selective_scan_fwd(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                                    const float *Dskip, const void *z, const float *dt_bias, const float *h0,
                                    const int *lengths, void *y, float *h_final,
                                    void *workspace, size_t workspace_bytes,
                                    int B, int T, int D, int N, int G, int softplus, kda_dtype_t dtype,
                                    void *stream);

/*
 * kda_selective_scan_step -- one token per sequence: x, dt, z, y [B, D],
 * Bm, Cm [B, G, N], the states h [B, D, N] float32 advanced IN PLACE.
 */
kda_status_t kda_selective_scan_step(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                                     const float *Dskip, const void *z, const float *dt_bias, float *h, void *y,
                                     int B, int D, int N, int G, int softplus, kda_dtype_t dtype, void *stream);

/*
 * kda_selective_scan_bwd -- gradients of kda_selective_scan_fwd for the
 * upstream gradients dy [B, T, D] (dtype) of y and dh_final [B, D, N] (float32,
 * or NULL) of h_final; the states are recomputed, nothing of the forward call
 * is needed.
 *
 *   dx, ddt [B, T, D] dtype;  dz [B, T, D] dtype, NULL exactly when z is NULL
 *   dA [D, N] float32;  dBm, dCm [B, T, G, N] dtype
 *   dDskip [D] float32, NULL exactly when Dskip is NULL
 *   ddt_bias [D] float32, NULL exactly when dt_bias is NULL
 *   dh0 [B, D, N] float32 or NULL (not written)
 */
size_t kda_selective_scan_bwd_workspace_bytes(int B, int T, int D, int N, int G);

kda_status_t kda_selective_scan_bwd(const void *dy, const void *x, const void *dt, const float *A, const void *Bm,
                                    const void *Cm, const float *Dskip, const void *z, const float *dt_bias,
                                    const float *h0, const float *dh_final, const int *lengths,
                                    void *dx, void *ddt, float *dA, void *dBm, void *dCm, float *dDskip, void *dz,
                                    float *ddt_bias, float *dh0, void *workspace, size_t workspace_bytes,
                                    int B, int T, int D, int N, int G, int softplus, kda_dtype_t dtype,
                                    void *stream);

/*
 * kda_layer_norm_fwd -- y = (x - mean) / sqrt(var + eps) * weight + bias over
 * rows of D channels, the variance over D (not D - 1).
 *
 *   x, y   [rows, D] dtype; y may be x itself
 *   weight [D] float32 or NULL (1), bias [D] float32 or NULL (0)
 *   eps    >= 0, finite.  With eps = 0 a row of one value has no defined result (0 / 0
 *          by the formula; NaN, or what rounding leaves of the mean, magnified)
 *
 * Centred values are squared in float32: their squares' sum has to stay below its
 * 3.4e38 (beyond, the variance is infinite and y is bias).
 *
 * D from 1 to 16384 (KDA_ERR_UNSUPPORTED beyond), rows below 2^40.
 */
kda_status_t kda_layer_norm_fwd(const void *x, const float *weight, const float *bias, float eps, void *y,
                                int64_t rows, int D, kda_dtype_t dtype, void *stream);

/*
 * kda_layer_norm_bwd -- gradients of kda_layer_norm_fwd: dx [rows, D] (dtype;
 * may be dy itself), dweight and dbias [D] float32, each or both NULL where
 * not wanted.  The rows' means and variances are computed again from x.
 */
size_t kda_layer_norm_bwd_workspace_bytes(int64_t rows, int D);

kda_status_t kda_layer_norm_bwd(const void *dy, const void *x, const float *weight, float eps, void *dx,
                                float *dweight, float *dbias, void *workspace, size_t workspace_bytes,
                                int64_t rows, int D, kda_dtype_t dtype, void *stream);

/*
 * The softmax attention layers between recurrent ones: a serving step's plan,
 * norm and rotation of queries and keys, a paged cache in 8 bits and the
 * attention that reads it.  Common to these calls:
 *
 *  - The cache of one layer is
 *      k_codes [pages, Hk, page, D]   one byte each
 *      v_codes [pages, Hk, D, page]   one byte each, tokens innermost
 *      k_scale, v_scale [pages, Hk]   float32
 *    A value is its code (kda_code_t) times the scale of its page and head,
 *    which is not negative.
 *    page (tokens a page) is 16, 32, 64 or 128, D is 64, 128 or 256
 *    (KDA_ERR_UNSUPPORTED otherwise); pages * page below 2^31, the codes below
 *    2^40 bytes.  A fresh cache needs no initialisation.
 *  - Slot s of the cache is place s % page of page s / page.
 *  - block_table [B, max_pages] int32 holds each sequence's pages in order;
 *    entries behind its last page are not read.
 *  - Numbers on the device (lengths, tables, slots, row starts) are not seen by
 *    the host.  Whatever they hold, no call reads or writes outside its
 *    buffers: what names no place of them is skipped, as stated.
 *  - Token rows q, k, v hold heads of D channels, heads next to each other;
 *    where strides are given (elements from one token to the next, at least a
 *    row) they may be parts of a wider matrix, such as a fused projection, and
 *    need only be aligned to their element.  int32 and scale buffers are
 *    aligned to 4 bytes.
 *  - dtype (KDA_F32 or KDA_BF16) is the type of the token rows.  Arithmetic and
 *    sums are float32, but for the weights of the attention (stated there); each
 *    output is rounded once, when stored.
 *  - Workspaces and overlaps as for the calls above.
 */

/*
 * kda_cache_plan -- what a serving step needs to know of its requests, built on
 * the device: request b has cached[b] tokens in the cache and brings added[b].
 *
 *   cached, added [B] int32
 *   block_table   [B, max_pages] int32: entries of the cached tokens' pages are
 *                 read, those of pages that the new tokens begin are written
 *   free_pages    [free_capacity] int32, free_count [1] int32 (clamped to the
 *                 capacity): a list of free pages, taken from its end, for request
 *                 0 first
 *   q_start       [B + 1] int32: each request's first row among the step's tokens
 *   context       [B] int32: its tokens after the step
 *   positions     [tokens] int32: each row's place in its sequence
 *   slots         [tokens] int32: and in the cache
 *   free_left     [1] int32: entries of free_pages that are still free (not free_count itself)
 *
 * Requests are served in order, while the free pages and the `tokens` rows last
 * for them and all before them.  One that is not served (nor one with a negative
 * length, or more pages than the table holds, which takes none) keeps its rows,
 * but its context is 0, its rows' positions and slots are -1, and its table is
 * left as it is.  Rows behind the last request have positions and slots -1;
 * q_start does not pass `tokens`.  A row whose page has a number that is negative,
 * or makes a slot of 2^31 or more, has slot -1.
 */
kda_status_t kda_cache_plan(const int *cached, const int *added, int *block_table, const int *free_pages,
                            const int *free_count, int *q_start, int *context, int *positions, int *slots,
                            int *free_left, int B, int max_pages, int free_capacity, int tokens, int page, void *stream);

/*
 * kda_qk_norm_rope_fwd -- norm of each query and key head and rotation by the
 * token's position, in one pass:
 *
 *   n = x / sqrt(mean_d x^2 + eps) * weight
 *   y = n with the pairs of its first rotary_dim channels turned by the angles
 *       of the token's row of `rotary`: (a, b) -> (a cos - b sin, a sin + b cos)
 *
 *   q, q_out [tokens, Hq, D] dtype, k, k_out [tokens, Hk, D] dtype, with strides;
 *            an output may be its own input
 *   q_weight, k_weight [D] float32, each or both NULL (ones)
 *   eps      >= 0, finite.  With eps = 0 a row of zeros is NaN
 *   rotary   [rotary_rows, rotary_dim] float32, rotary_dim / 2 cosines and then as
 *            many sines a row; NULL with rotary_dim = 0: no rotation
 *   positions [tokens] int32, the rows of `rotary` to use; NULL, if there is none:
 *            every row is a token.  A negative one marks a row of no token: its input
 *            is not read, its output is zero.  One of rotary_rows or more makes its
 *            outputs NaN, with a table
 *   neighbours  0: the pairs are (i, i + rotary_dim / 2); otherwise (2 i, 2 i + 1)
 *
 * D even, up to 512, rotary_dim even, up to D.  A head's sum of squares has to
 * stay below float32's 3.4e38, and its mean with eps, unless 0, not below 1.2e-38.
 */
kda_status_t kda_qk_norm_rope_fwd(const void *q, const void *k, const float *q_weight, const float *k_weight, float eps,
                                  const int *positions, const float *rotary, void *q_out, void *k_out,
                                  int64_t tokens, int Hq, int Hk, int D, int rotary_dim, int rotary_rows, int neighbours,
                                  int64_t q_stride, int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride,
                                  kda_dtype_t dtype, void *stream);

/*
 * kda_qk_norm_rope_bwd -- its gradients: dq [tokens, Hq, D] and dk [tokens, Hk, D]
 * (dtype; each may be its upstream gradient dq_out or dk_out, or its input q or k,
 * with the same stride), dq_weight and
 * dk_weight [D] float32, summed over tokens and heads, each or both NULL where
 * not wanted (a workspace is needed for them only).  q and k are the forward's
 * inputs.  Rows of a negative position have zero gradients and add nothing;
 * rows of one beyond the table make theirs, and the weights', NaN.
 */
size_t kda_qk_norm_rope_bwd_workspace_bytes(int64_t tokens, int Hq, int Hk, int D);

kda_status_t kda_qk_norm_rope_bwd(const void *dq_out, const void *dk_out, const void *q, const void *k,
                                  const float *q_weight, const float *k_weight, float eps,
                                  const int *positions, const float *rotary, void *dq, void *dk,
                                  float *dq_weight, float *dk_weight, void *workspace, size_t workspace_bytes,
                                  int64_t tokens, int Hq, int Hk, int D, int rotary_dim, int rotary_rows, int neighbours,
                                  int64_t dq_out_stride, int64_t dk_out_stride, int64_t q_stride, int64_t k_stride,
                                  int64_t dq_stride, int64_t dk_stride, kda_dtype_t dtype, void *stream);

/*
 * kda_cache_append -- new keys and values into the cache, IN PLACE.
 *
 *   k, v   [tokens, Hk, D] dtype, with strides
 *   slots  [tokens] int32; tokens whose slot is outside the cache are skipped
 *
 * For each page and head that tokens go to, with Q the largest code (448 or 127):
 *   scale' = max(scale, largest |new| * (1 / Q)), or the second alone where the
 *            first place written is the page's first (it starts anew, whatever
 *            it and its scale held)
 *   code   = new / scale' to the nearest code, ties to even
 *   codes in front of the first place written: code * (scale / scale') to the
 *            nearest code, where the scale grew; all other places are left as they are
 * in float32.  Infinities and NaN leave the scale not finite: such a page and
 * head reads as NaN until it starts anew.
 *
 * The tokens of a call that go to one page stand next to each other in the call, in
 * any order, as those of one sequence do: no token of another page and none that is
 * skipped comes between them (each such part would be taken for all of them, at
 * once).  Of two with the same slot the later one counts.  A page that two sequences
 * share is not written by either.
 */
kda_status_t kda_cache_append(const void *k, const void *v, const int *slots, void *k_codes, void *v_codes,
                              float *k_scale, float *v_scale, int tokens, int Hk, int D, int pages, int page,
                              int64_t k_stride, int64_t v_stride, kda_code_t code, kda_dtype_t dtype, void *stream);

/*
 * kda_cache_attention -- causal attention over the cache: each query head reads
 * key and value head (its number) / (Hq / Hk).
 *
 *   o = sum_t softmax_t(scale q . K[t]) V[t],  lse = log sum_t exp(scale q . K[t])
 *
 *   q, out  [tokens, Hq, D] dtype, contiguous, all sequences' rows together
 *   q_start [B + 1] int32: sequence b has rows q_start[b] to q_start[b + 1] - 1, not
 *           descending, clamped to [0, tokens]; NULL: one row each (tokens = B)
 *   context [B] int32: its tokens in the cache, those of the rows among them
 *           (clamped to the table).  Row i of n stands at place context - n + i
 *           and sees the places up to its own
 *   lse     [tokens, Hq] float32, or NULL
 *   max_queries  rows of the longest sequence, as far as the host knows: chooses
 *           the kernel, and the results are right for any value (taken as at least 1
 *           and at most tokens)
 *
 * For their product with the values, the weights are rounded to float16 with 11 bits
 * (float32 rows: two parts, 22 bits) relative to the row's largest weight x value
 * scale, and lose bits only where that is 2^27 times smaller; their sum is of float32
 * ones.  A value scale below 1.2e-38 counts as 0.
 *
 * A page and head whose scale is not finite makes the rows that see its tokens
 * NaN.  Pages whose table entry names none of the cache (such as -1, for a page
 * that was given up) are not seen.  A row that sees no place has out 0 and lse -inf.
 * Rows of no sequence are left as they were.
 *
 * tokens * Hq below 2^31.  The units of work (64 places of the table x key head x
 * block of 16 or more query rows of a head's group) of a call whose sequences have
 * few rows have to stay below 2^31 too (KDA_ERR_UNSUPPORTED beyond).  Row starts that
 * descend may count some rows many times: what such a call writes is inside its
 * outputs, and nothing where they count 2^31 units or more.
 */
size_t kda_cache_attention_workspace_bytes(int tokens, int B, int Hq, int Hk, int D, int page, int max_pages,
                                           int max_queries);

kda_status_t kda_cache_attention(const void *q, const void *k_codes, const void *v_codes, const float *k_scale,
                                 const float *v_scale, const int *block_table, const int *context, const int *q_start,
                                 void *out, float *lse, void *workspace, size_t workspace_bytes,
                                 int tokens, int B, int Hq, int Hk, int D, int pages, int page, int max_pages,
                                 int max_queries, float scale, kda_code_t code, kda_dtype_t dtype, void *stream);

/* Static, human-readable name of a status code (never NULL). */
const char *kda_status_string(kda_status_t status);   /* codes outside the set: "KDA_ERR_UNKNOWN" */

/* KDA_ABI_VERSION of the built library. */
int kda_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
