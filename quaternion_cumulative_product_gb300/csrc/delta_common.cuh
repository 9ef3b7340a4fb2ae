// delta_common.cuh -- what the kernels of the gated delta rule over whole
// sequences share: arguments, sequence and chunk geometry, decays.
//
// Chunked form.  A chunk holds C = 64 steps; M enters it, M' leaves it, and with
// the decay sums G_t = g_0 + .. + g_t inside the chunk, D_ts = exp(G_t - G_s):
//
//     A_ts = D_ts <k_t, k_s>  (s < t)        P_ts = scale D_ts <q_t, k_s>  (s <= t)
//     e_t  = v_t - exp(G_t) M^T k_t - sum_s A_ts beta_s e_s        (a triangular system)
//     u_t  = beta_t e_t
//     o_t  = scale exp(G_t) M^T q_t + sum_s P_ts u_s
//     M'   = exp(G_C) M + sum_t exp(G_C - G_t) k_t u_t^T
//
// Backward, from the cotangents do_t and dM' (d_final at the end):
//
//     w_t  = exp(G_C - G_t) dM'^T k_t + sum_{s>=t} P_st do_s - sum_{s>t} A_st beta_s w_s
//     dM   = exp(G_C) dM' + sum_t exp(G_t) (scale q_t do_t^T - k_t (beta_t w_t)^T)
//     dv_t = beta_t w_t            dbeta_t = <e_t, w_t>
//     X_ts = scale D_ts <do_t, u_s> (s <= t)       Y_ts = -D_ts <dv_t, u_s>  (s < t)
//     dq_t = scale exp(G_t) M do_t + sum_s X_ts k_s
//     dk_t = row_t + col_t
//     row_t = -exp(G_t) M dv_t + sum_s Y_ts k_s
//     col_t = exp(G_C - G_t) dM' u_t + sum_s X_st q_s + sum_s Y_st k_s
//     dg_t  = sum_{r>=t>s} Z_rs + sum_{r>=t} a_r + sum_{s<t} b_s + exp(G_C) <M, dM'>
//     Z_rs  = X_rs <q_r, k_s> + Y_rs <k_r, k_s>   (s < r)
//     a_r   = exp(G_r) (scale <q_r, M do_r> - <k_r, M dv_r>)
//     b_s   = exp(G_C - G_s) <k_s, dM' u_s>
//
// (dg_t holds what crosses step t, from a state or key before it to a query, key or state
// from it on: each term has the factor exp(g_t), and where that is zero so is dg_t.  The same
// sum by way of the G's gradients, <q, dq> + <k, row - col> from step t on, adds and takes
// off every pair inside the rest of the chunk, and what is left of their rounding can be far
// larger than the gradient of a strong decay.)
//
// (w is kept rather than dv, so that beta = 0 loses nothing.)
#pragma once

#include "mixer_device.cuh"
#include "quat_common.cuh"
#include "quat_host.h"
#include "quat_mixer.h"

namespace qs {

constexpr int DC = QS_DELTA_STEPS;   // steps per chunk
constexpr int kMostOrdered = 128;   // packed sequences that are put in order of length

struct DeltaArgs {
    const void *q, *k, *v, *g, *beta;
    const float *init;
    void *o;
    float *fin, *carries, *errors;
    // backward
    const float *carries_in, *errors_in, *d_final;
    const void *d_o;
    void *dq, *dk, *dv, *dg, *dbeta;
    float *d_init;
    float *ds;        // dM' of every chunk [slots, Hv, Dk, Dv]
    float *w;         // w_t [B, S, Hv, Dv]
    float *dqh, *dkh; // dq, dk of every value head [B, S, Hv, Dk] (shared key heads)
    qsh::Strides sq, sk, sv;
    const int *offsets;
    long long B, S, N, NC, slots;   // NC: chunks per sequence without offsets
    // A sequence cut into segments (few sequences, long ones): segments, chunks in each;
    // the state that enters each segment (backward: the cotangent of the one that leaves
    // it) [N, Hv, segs, Dk, Dv]; a segment's own part and its map, [.., Dk, Dv] and [.., Dk, Dk].
    int segs;
    long long seg_chunks;
    const float *seg_m;
    float *seg_own, *seg_map;
    int Hk, Hv, Dk, Dv;
    int sms;   // of the device
    bool gate16;
    bool longest_first;   // packed sequences are walked in order of length
    float scale;
    Control ctl;
};

// One sequence: batch entry, first step, length, first carry slot.
struct Seq {
    long long b, s0, len, slot0;
};

__device__ __forceinline__ Seq seq_of(const DeltaArgs &a, long long n) {
    if (!a.offsets) return {n, 0, a.S, n * a.NC};
    const long long lo = a.offsets[n], hi = a.offsets[n + 1];
    const long long s0 = lo < 0 ? 0 : lo > a.S ? a.S : lo;
    const long long s1 = hi < s0 ? s0 : hi > a.S ? a.S : hi;
    return {0, s0, s1 - s0, s0 / DC + n};
}

// Segment `seg` of a sequence.
__device__ __forceinline__ Seq segment_of(const DeltaArgs &a, const Seq &s, int seg) {
    const long long c0 = seg * a.seg_chunks, off = c0 * DC, most = a.seg_chunks * DC;
    const long long left = s.len > off ? s.len - off : 0;
    return {s.b, s.s0 + off, left < most ? left : most, s.slot0 + c0};
}

// The sequence and chunk in a carry slot; false when the slot holds no chunk.
__device__ __forceinline__ bool chunk_of(const DeltaArgs &a, long long slot, Seq *seq, long long *chunk) {
    if (!a.offsets) {
        const long long n = slot / a.NC;
        *seq = seq_of(a, n);
        *chunk = slot - seq->slot0;
        return true;
    }
    long long lo = 0, hi = a.N;   // the last n with slot0(n) <= slot
    while (hi - lo > 1) {
        const long long mid = (lo + hi) / 2;
        if (seq_of(a, mid).slot0 <= slot) lo = mid;
        else hi = mid;
    }
    *seq = seq_of(a, lo);
    *chunk = slot - seq->slot0;
    return *chunk >= 0 && *chunk * DC < seq->len;
}

// Decay sums as a pair of floats (hi + lo): differences of sums far from zero
// keep the precision of their terms.
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ Sum2 sum2_add(const Sum2 a, const Sum2 b) {   // Knuth's two-sum
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = (a.hi - (s - t)) + (b.hi - t) + a.lo + b.lo;
    const float hi = s + e;
    return {hi, e - (hi - s)};
}

// A step's log decay.  Below -256 exp() is zero in fp32 by far, and so is every
// product of decays <= 1 over it: the clamp makes -inf (a cleared state) finite.
// In base-2 units, so that a decay is one exp2; the factor log2(e) rounds once, which
// is 2^-24 of the decay's logarithm, as a rounding of the gate itself would be.
__device__ __forceinline__ float clamp_gate(float g) { return (g < -256.f ? -256.f : g) * 1.4426950408889634f; }

// 2^x (the instruction: 2^-22 off at most).
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// exp(G_t - G_s) from sums kept in base-2 units.
__device__ __forceinline__ float decay(const Sum2 t, const Sum2 s) { return exp2_fast((t.hi - s.hi) + (t.lo - s.lo)); }

// Lanes 0..31 hold steps 2l and 2l+1: inclusive sums over the 64 steps.
__device__ __forceinline__ void chunk_sums(float g0, float g1, Sum2 *s0, Sum2 *s1) {
    const int lane = threadIdx.x % 32;
    Sum2 run = sum2_add({g0, 0.f}, {g1, 0.f});
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const Sum2 other = {__shfl_up_sync(0xffffffffu, run.hi, o), __shfl_up_sync(0xffffffffu, run.lo, o)};
        if (lane >= o) run = sum2_add(other, run);
    }
    Sum2 before = {__shfl_up_sync(0xffffffffu, run.hi, 1), __shfl_up_sync(0xffffffffu, run.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
    *s0 = sum2_add(before, {g0, 0.f});
    *s1 = run;
}

}  // namespace qs
