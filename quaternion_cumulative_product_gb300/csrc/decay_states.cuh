// decay_states.cuh -- linear attention in fp32: the states between chunks, all chunks at once.
//
// With the sums of delta_common.cuh, a chunk adds to the state that passes it
//
//     own = sum_t exp(G_C - G_t) k_t v_t^T          (backward, to the cotangent: sum_t scale exp(G_t) q_t do_t^T)
//
// whatever that state is: a kernel for the chunks' own parts, one that runs along the chunks
// of each (sequence, head), element by element.  (The delta rule's states have to be walked.)
//
// Bound: own, fp32 arithmetic (64 x 128 x 128 a chunk; 8 x 8 values of a product per thread, two
// 16-byte reads of shared memory a side for 64 multiply-adds: 127 us for 2048 chunks of 128, 45% of
// the fp32 rate); the run, memory (36 us there, 268 MB, 7.4 TB/s).
#pragma once

#include "delta_prep.cuh"

namespace qs {

// One direction; the backward takes both in one launch.
struct StateSide {
    float *states;        // [slots, Hv, Dk, Dv]: the chunks' own parts, then the state that enters each (rev: the cotangent of the one that leaves it)
    const float *first;   // state that enters the first chunk (rev: cotangent that leaves the last) [N, Hv, Dk, Dv], or NULL
    float *last;          // what the run ends with, or NULL
    bool rev;
};

struct StateArgs {
    DeltaArgs d;
    float *whole;         // [slots, Hv]
    StateSide side[2];
    bool cut_only;        // of the sequences that are cut only
};

constexpr int kOwnThreads = 256;

// D: 64 or 128, at least Dk and Dv.
template <int D>
__global__ void __launch_bounds__(kOwnThreads) decay_own_kernel(const __grid_constant__ StateArgs s) {
    extern __shared__ __align__(16) float rows[];   // [64][D] k (q), [64][D] v (dO)
    __shared__ ChunkGates gt;
    const DeltaArgs &a = s.d;
    const bool rev = s.side[blockIdx.y].rev;
    let_next_start();
    const int head = blockIdx.x % a.Hv, kh = head / (a.Hv / a.Hk), tid = threadIdx.x;
    const long long slot = blockIdx.x / a.Hv;
    Seq seq;
    long long c;
    if (!chunk_of(a, slot, &seq, &c) || (s.cut_only && !is_cut(a, seq))) return;
    const long long t0 = c * DC;
    const int left = (int)min((long long)DC, seq.len - t0);
    if (tid < 32) warp_gates(gt, read_gates<false>(a, seq, t0, head));
    __syncthreads();
    float *x = rows, *y = rows + DC * D;
    const qsh::Strides so = {(long long)a.S * a.Hv * a.Dv, (long long)a.Hv * a.Dv, a.Dv};
    const qsh::Strides &sx = rev ? a.sq : a.sk, &sy = rev ? so : a.sv;
    const float *px = static_cast<const float *>(rev ? a.q : a.k) + seq.b * sx.b + (seq.s0 + t0) * sx.s + (long long)kh * sx.h;
    const float *py = static_cast<const float *>(rev ? a.d_o : a.v) + seq.b * sy.b + (seq.s0 + t0) * sy.s + (long long)head * sy.h;
    for (int i = tid; i < DC * D / 4; i += kOwnThreads) {
        const int r = i / (D / 4), col = i % (D / 4) * 4;
        float4 u = q_zero(), v = q_zero();
        if (r < left && col < a.Dk) {
            const float f = rev ? a.scale * gt.grown[r] : gt.left[r];
            u = load4(px + r * sx.s + col);
            u = make_float4(u.x * f, u.y * f, u.z * f, u.w * f);
        }
        if (r < left && col < a.Dv) v = load4(py + r * sy.s + col);
        store4(x + r * D + col, u), store4(y + r * D + col, v);
    }
    __syncthreads();
    // A thread: rows 4 i .. and 4 i + D / 2 .. of dk, columns likewise of dv, T of each.
    constexpr int T = D / 16, H = T / 4;   // 8 (two quads) or 4 (one)
    const int i0 = tid / 16 * 4, j0 = tid % 16 * 4;
    float2 m[T][T / 2];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T / 2; ++j) m[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int t = 0; t < DC; ++t) {
        float4 u[H], v[H];
#pragma unroll
        for (int h = 0; h < H; ++h) u[h] = *reinterpret_cast<const float4 *>(x + t * D + h * 64 + i0), v[h] = *reinterpret_cast<const float4 *>(y + t * D + h * 64 + j0);
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const float4 &q = u[i / 4];
            const float f = i % 4 == 0 ? q.x : i % 4 == 1 ? q.y : i % 4 == 2 ? q.z : q.w;
#pragma unroll
            for (int j = 0; j < H; ++j) {
                m[i][2 * j] = fma2(make_float2(f, f), make_float2(v[j].x, v[j].y), m[i][2 * j]);
                m[i][2 * j + 1] = fma2(make_float2(f, f), make_float2(v[j].z, v[j].w), m[i][2 * j + 1]);
            }
        }
    }
    float *out = s.side[blockIdx.y].states + (size_t)blockIdx.x * a.Dk * a.Dv;
#pragma unroll
    for (int i = 0; i < T; ++i) {
        const int r = i / 4 * 64 + i0 + i % 4;
        if (r < a.Dk)
#pragma unroll
            for (int j = 0; j < H; ++j)
                if (j * 64 + j0 < a.Dv) store4(out + (size_t)r * a.Dv + j * 64 + j0, make_float4(m[i][2 * j].x, m[i][2 * j].y, m[i][2 * j + 1].x, m[i][2 * j + 1].y));
    }
    if (tid == 0 && blockIdx.y == 0) s.whole[blockIdx.x] = gt.whole;
}

// A thread per four values of a (sequence, head); eight chunks' parts on their way at a time.
__global__ void __launch_bounds__(256) decay_run_kernel(const __grid_constant__ StateArgs s, unsigned parts) {
    const DeltaArgs &a = s.d;
    const StateSide &side = s.side[blockIdx.y];
    wait_for_last();
    const size_t size = (size_t)a.Dk * a.Dv, e = ((size_t)(blockIdx.x % parts) * 256 + threadIdx.x) * 4, nh = blockIdx.x / parts;
    if (e >= size) return;
    const Seq seq = seq_of(a, (long long)(nh / a.Hv));
    const int head = (int)(nh % a.Hv), chunks = (int)((seq.len + DC - 1) / DC);
    if (s.cut_only && !is_cut(a, seq)) return;
    auto at = [&](int i) { return (size_t)(seq.slot0 + (side.rev ? chunks - 1 - i : i)) * a.Hv + head; };
    float4 m = side.first ? __ldg(reinterpret_cast<const float4 *>(side.first + nh * size + e)) : q_zero();
    constexpr int AHEAD = 8;
    for (int i0 = 0; i0 < chunks; i0 += AHEAD) {
        float4 own[AHEAD];
        float f[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (i0 + k < chunks) own[k] = *reinterpret_cast<const float4 *>(side.states + at(i0 + k) * size + e), f[k] = s.whole[at(i0 + k)];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (i0 + k < chunks) {
                *reinterpret_cast<float4 *>(side.states + at(i0 + k) * size + e) = m;
                m = make_float4(fmaf(f[k], m.x, own[k].x), fmaf(f[k], m.y, own[k].y), fmaf(f[k], m.z, own[k].z), fmaf(f[k], m.w, own[k].w));
            }
    }
    if (side.last) *reinterpret_cast<float4 *>(side.last + nh * size + e) = m;
}

}  // namespace qs
