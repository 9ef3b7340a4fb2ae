/*
 * quat_mixer.h -- C ABI of the sequence-mixer operators around the quaternion
 * scan: the per-head norm of queries and keys with their rotation by the
 * cumulative quaternion, and the gated delta rule (whole sequences, its
 * backward, and single tokens on a pool of states).
 *
 * Conventions are those of quat_cumprod.h: plain device pointers on the current
 * device, 16-byte aligned, caller-owned; `stream` is a cudaStream_t; every call
 * validates its arguments, enqueues its work on `stream` and returns; scratch
 * is the library's workspace of the (device, stream) (a call that needs more of
 * it allocates and synchronizes, and returns QS_ERR_NOMEM while the stream is
 * being captured); a device-side wait that runs out is reported by
 * quat_cumprod_status(); outputs must not overlap inputs (quat_delta_step's
 * state is updated in place).  Status codes are quat_cumprod.h's.
 *
 * quat_cumprod_debug_stall_tile(k) makes CTA k of quat_delta_fwd's and _bwd's and
 * of quat_decay_fwd's and _bwd's bfloat16 walks wait for rows that never come, as it
 * does a tile of the scan.
 *
 * Element types: QS_F32 or QS_BF16.  Sums, norms and states are fp32.  The delta rule's
 * products leave out at most 2^-24 of a product, or, where only bfloat16 outputs are made
 * of them, 2^-15 (rms 2^-17); its decays are off by 2^-22 and by 2^-24 of their logarithm
 * at most.  (fp32 values past 2^128 - 2^119 count as infinite there.)  An output in bfloat16 is rounded to nearest even once, when stored.
 *
 * Strides: a `strides` argument holds, for each tensor it names, the distances
 * in elements between batch entries, between steps and between heads (three
 * int64 each); the last dimension is contiguous.  NULL means contiguous.  Each
 * stride must be a multiple of 16 bytes and not negative.
 */
#ifndef QUAT_MIXER_H
#define QUAT_MIXER_H

#include <stdint.h>

#include "quat_cumprod.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { QS_F32 = 0, QS_BF16 = 1 };            /* element types               */
enum { QS_NORM_RMS = 0, QS_NORM_L2 = 1 };    /* norms of quat_norm_rotate_* */

/* Steps per chunk of the delta rule's carries (the scan's QS_CARRY_STEPS). */
#define QS_DELTA_STEPS 64
/* Largest head dimension of the calls below. */
#define QS_ROTATE_MAX_D 256
#define QS_DELTA_MAX_D 128

/*
 * Norm and rotation of queries and keys.  For every head vector x [D] of
 * q [B,S,Hq,D] and k [B,S,Hk,D]:
 *
 *     n = x * (sum(x^2) / (RMS ? D : 1) + eps)^(-1/2) * w        (w_q or w_k, fp32 [D]; NULL: 1)
 *     z_j = conj(cum_j) (x) n_j      j < J, n_j = n[4j .. 4j+3] as a quaternion [w,x,y,z]
 *     z   = n                        from 4J on
 *
 * with cum [B,S,H,J,4] (the scan's output, `cum_dtype`) of rotation head
 * h / (Hq/H) for query head h, h / (Hk/H) for key head h.  With unit
 * quaternions the inner product of two rotated vectors depends on the relative
 * rotation alone: <conj(c_t) (x) a, conj(c_s) (x) b> = <a, q_t .. q_{s+1} (x) b>
 * for cum[t] = q_t (x) cum[t-1], which is what a rotary position embedding
 * needs.  (That identity fails for c (x) a: the product does not commute.)
 * Requires Hq and Hk multiples of H, 4J <= D, D a multiple of 4, at most
 * QS_ROTATE_MAX_D (a multiple of 8 above 128).  `strides` names q, k.
 * Outputs are contiguous.
 */
int quat_norm_rotate_fwd(int dtype, int cum_dtype, int norm, float eps,
                         const void *q, const void *k, const void *cum, const float *w_q, const float *w_k,
                         void *q_out, void *k_out, const int64_t *strides,
                         int64_t B, int64_t S, int64_t H, int64_t J, int64_t Hq, int64_t Hk, int64_t D,
                         void *stream);

/*
 * Its vector-Jacobian product for cotangents d_q_out, d_k_out (contiguous),
 * recomputed from the inputs: d_q, d_k (contiguous, `dtype`), d_cum
 * [B,S,H,J,4] (`cum_dtype`; the sum over the heads that share a rotation) and,
 * for weights given, d_w_q, d_w_k (fp32 [D]; the sum over all rows, in a fixed
 * order).  `strides` names q, k.
 */
int quat_norm_rotate_bwd(int dtype, int cum_dtype, int norm, float eps,
                         const void *q, const void *k, const void *cum, const float *w_q, const float *w_k,
                         const void *d_q_out, const void *d_k_out,
                         void *d_q, void *d_k, void *d_cum, float *d_w_q, float *d_w_k, const int64_t *strides,
                         int64_t B, int64_t S, int64_t H, int64_t J, int64_t Hq, int64_t Hk, int64_t D,
                         void *stream);

/*
 * Gated delta rule over whole sequences.  For every value head h (with key head
 * h / (Hv/Hk)) a state M [Dk,Dv] runs along the sequence:
 *
 *     M~_t = exp(g_t) M_{t-1}
 *     e_t  = v_t - M~_t^T k_t
 *     M_t  = M~_t + k_t (beta_t e_t)^T
 *     o_t  = scale * M_t^T q_t
 *
 * q, k [B,S,Hk,Dk], v, o [B,S,Hv,Dv] (`dtype`), g, beta [B,S,Hv] (`gate_dtype`,
 * contiguous; g <= 0, -inf clears the state), init and final_state
 * [N,Hv,Dk,Dv] fp32 (init NULL: zeros; final_state NULL: not written).
 * Sequences: N = B without `offsets`; with offsets (int32 [N+1] on the device,
 * offsets[0] = 0, not decreasing, offsets[N] = S) B is 1 and sequence n holds
 * the steps offsets[n] .. offsets[n+1]-1.  Empty sequences keep their state.
 * Steps are taken 64 at a time: a NaN or infinity at a step spoils the outputs
 * of its sequence from the start of its chunk on (never another sequence's).
 * For a backward, `carries` and `errors` (both or neither) also receive the
 * state entering every QS_DELTA_STEPS-step chunk and the e_t:
 *     carries  fp32 [B, ceil(S/64), Hv, Dk, Dv]; with offsets [S/64 + N, Hv, Dk, Dv],
 *              chunk c of sequence n in slot offsets[n]/64 + n + c
 *     errors   fp32 [B, S, Hv, Dv]
 * `strides` names q, k, v (in bfloat16 none may be zero over more than one entry).
 * Requires Hv a multiple of Hk, Dk and Dv multiples of 8 up to QS_DELTA_MAX_D.
 */
int quat_delta_fwd(int dtype, int gate_dtype, float scale,
                   const void *q, const void *k, const void *v, const void *g, const void *beta, const float *init,
                   void *o, float *final_state, float *carries, float *errors,
                   const int64_t *strides, const int32_t *offsets, int64_t N,
                   int64_t B, int64_t S, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, void *stream);

/*
 * Its vector-Jacobian product from the carries and errors of the forward, for
 * cotangents d_o (contiguous, `dtype`) and d_final (fp32, NULL: zeros): d_q,
 * d_k, d_v (`dtype`; the first two summed over the value heads that share a key
 * head), d_g, d_beta (`gate_dtype`), d_init (fp32, NULL: not written).  d_g is
 * exactly zero where exp(g) is zero in fp32.  Sums run in a fixed order.
 */
int quat_delta_bwd(int dtype, int gate_dtype, float scale,
                   const void *q, const void *k, const void *v, const void *g, const void *beta,
                   const float *carries, const float *errors, const void *d_o, const float *d_final,
                   void *d_q, void *d_k, void *d_v, void *d_g, void *d_beta, float *d_init,
                   const int64_t *strides, const int32_t *offsets, int64_t N,
                   int64_t B, int64_t S, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, void *stream);

/*
 * Gated delta rule for T new tokens (usually one) of each of N sequences, on
 * states that stay in a pool: state [P,Hv,Dk,Dv] fp32, updated in place.  Row n
 * uses state slots[n] (int32 [N] on the device; NULL: slot n); a slot outside
 * 0 .. P-1 marks an idle row, whose o is zero and which touches no state.  Two
 * rows must not name the same slot.  q, k [N,T,Hk,Dk], v, o [N,T,Hv,Dv], g,
 * beta [N,T,Hv]; `strides` names q, k, v.
 */
int quat_delta_step(int dtype, int gate_dtype, float scale,
                    const void *q, const void *k, const void *v, const void *g, const void *beta,
                    float *state, const int32_t *slots, void *o, const int64_t *strides,
                    int64_t P, int64_t N, int64_t T, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, void *stream);

/*
 * Linear attention with a decay for each head, over whole sequences.  For every
 * value head h (with key head h / (Hv/Hk)) a state M [Dk,Dv] runs along the sequence:
 *
 *     M_t = exp(g_t) M_{t-1} + k_t v_t^T
 *     o_t = scale * M_t^T q_t
 *
 * Tensors, sequences, strides and sizes are those of quat_delta_fwd (without beta);
 * init NULL: zeros, final_state NULL: not written.  A NaN or infinity at a step
 * spoils the outputs of its sequence from the start of its chunk (at most 128 steps)
 * on, never another sequence's.  With offsets, rows from offsets[N] on (where that is
 * less than S) are not used, and left as they were in every output.
 *
 * Precision: as the delta rule (o, d_q, d_k and d_v in bfloat16 leave out 2^-17 of a
 * product; states and fp32 outputs 2^-24).  d_g leaves out 2^-24 of a product, with bfloat16
 * gates 2^-17.
 */
int quat_decay_fwd(int dtype, int gate_dtype, float scale,
                   const void *q, const void *k, const void *v, const void *g, const float *init,
                   void *o, float *final_state, const int64_t *strides, const int32_t *offsets, int64_t N,
                   int64_t B, int64_t S, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, void *stream);

/*
 * Its vector-Jacobian product, recomputed from the inputs, for cotangents d_o
 * (contiguous, `dtype`) and d_final (fp32, NULL: zeros): d_q, d_k (`dtype`; summed over
 * the value heads that share a key head), d_v (`dtype`), d_g (`gate_dtype`; exactly zero
 * where exp(g) is zero in fp32), d_init (fp32, NULL: not written).  Sums run in a fixed
 * order.  Scratch: the states between chunks.
 */
int quat_decay_bwd(int dtype, int gate_dtype, float scale,
                   const void *q, const void *k, const void *v, const void *g, const float *init,
                   const void *d_o, const float *d_final,
                   void *d_q, void *d_k, void *d_v, void *d_g, float *d_init,
                   const int64_t *strides, const int32_t *offsets, int64_t N,
                   int64_t B, int64_t S, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, void *stream);

/* The same recurrence for T new tokens (usually one) of each of N sequences, on a pool of states, as quat_delta_step. */
int quat_decay_step(int dtype, int gate_dtype, float scale,
                    const void *q, const void *k, const void *v, const void *g,
                    float *state, const int32_t *slots, void *o, const int64_t *strides,
                    int64_t P, int64_t N, int64_t T, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QUAT_MIXER_H */
