// decay_walk.cuh -- linear attention with a decay on the tensor cores, bfloat16: one walk over
// the chunks of a (sequence, head) that serves the forward and all three products of the backward.
//
// A walk takes "queries" x, "keys" y [.., dk] and "values" z [.., dv] and computes
//
//     out_t = scale sum_s D_ts <x_t, y_s> z_s,      D_ts = exp(|G_t - G_s|'s decay between s and t)
//
// over the steps s <= t (forward in time) or s >= t (backward in time):
//
//     o  = (q, k, v) forward          dq = (dO, v, k) forward
//     dv = (k, q, dO) backward        dk = (v, dO, q) backward
//
// Chunks hold C = 128 steps.  With the state M [dk][dv] that enters a chunk (from earlier steps
// forward, later ones backward) and the decay sums G_t = g_0 + .. + g_t inside the chunk:
//
//     out = f (x M) + P z,            P_ts = scale D_ts <x_t, y_s>,     f_t = scale exp(G_t) | exp(G_C - G_t)
//     M'  = exp(G_C) M + y^T (h z),                                     h_s = exp(G_C - G_s) | scale exp(G_s)
//
// (forward | backward in time: backward, M is the state's cotangent).  Nothing but M' = exp(G_C) M + .. links two chunks, and that is a
// sum in registers: the tensor cores are kept busy across chunks by roles that run at the same time:
//
//     state    two warpgroups: M^T [dv][dk] in fp32 registers, one value row per thread, half of dk
//              each; M's terms to shared memory; the terms of the second half of h z; out to memory
//     convert  two warpgroups: the terms of the first half of h z; P from S = x y^T (in place, in tensor
//              memory); f Y and its products with `beside`
//     one warp each: products, copies (TMA into a ring of tiles), gates, stores
//
// Per chunk, in the order of issue: S, dM = (h z)^T y over the first 64 steps, Y = x M, dM over the
// other 64, out = f Y + P z.
//
// Terms (tensor_core.cuh): h z in three, so that states have fp32 precision (they add up rounded
// once a chunk).  P and the M of Y, of which only bfloat16 outputs are made, in two: at most 2^-17 of
// them is left out, far below the output's own rounding (one term each, 2^-8, would be as large as
// that: 2.3e-3 instead of 1.7e-3 from 64 bits, for 111 instead of 121 us forward).  Where Y
// goes into d_g as well (dots) M has a third one for fp32 gates (d_g is then 3e-7 to 6e-7 from 64
// bits, with two 2e-6).
//
// Measured, 8 x 4096 x 16 x 128 (128 walks of 32 chunks): forward 121 us (4.4 TB/s, 0.65 of a copy's rate),
// 3.7 us a chunk; dv 118, dq 174 and dk 193 us (they also write and read the states, 268 MB each).
// 1 x 131072 x 16 x 64 in 19 segments: 409 us, the sums 125 and the walk 277 of them.
// Bound: the products, beside the other roles' use of shared memory.  64 of 128 x 128 x 16 a chunk (S 8,
// Y 16, dM 24, P z 16) take 80 to 100 cycles each where they come in a row (64 at the peak rate); the rest is
// the way from one to the next: out, then the next chunk's S, then its P.
#pragma once

#include <type_traits>

#include <cuda_fp16.h>

#include "delta_prep.cuh"

namespace qs {

constexpr int WC = 128;              // steps per chunk
constexpr int kDecayThreads = 640;   // five warpgroups

struct DecayRole {
    CUtensorMap x, y, z, o, b;   // (o: of out, bfloat16; b: of `beside`)
    void *out;               // [B, S, Hv, dv], bfloat16 or (out32) fp32
    float *dots;             // <beside_t, f Y_t> [2][B, S, Hv] by halves of the columns
    const float *init;       // state that enters (first chunk of a walk) [N, Hv, ..], or NULL
    float *fin;              // state that leaves, or NULL
    float *dump;             // state that enters each chunk [slots, Hv, D * D], or NULL
    const float *other;      // another walk's states at the same places: cross = exp(G_C) <other, M>
    float *cross;            // [slots, Hv, 8]: a part for each warp of the state's
    const float *seg_m;      // state that enters each segment
    float *seg_own, *seg_decay;
    int gx, gy, gz, gb;      // value heads that share a head of x, y, z, beside
    int dk, dv;              // values of a row of x and y; of z and out
    int lane, col;           // distances in init and fin of the state's dv and dk
    bool out32;
};

struct DecayArgs {
    DecayRole role;
    const void *g;
    const int *offsets;
    long long B, S, N, NC, seg_chunks;   // NC: chunks per sequence without offsets
    int Hv, segs;
    bool gate16, longest_first;
    float scale;
    Control ctl;
};

// The state as the walks keep it between kernels: D * D floats, float4 j of (warpgroup, lane).
template <int D>
__device__ __forceinline__ size_t state_at(int j4, int wg, int lane) {
    return ((size_t)j4 * 2 * D + wg * D + lane) * 4;
}

struct __align__(16) WalkGates {
    float hi[WC];      // G_t = hi + lo, in base-2 units
    float mid[WC];     // decay between s and the end of its 32 steps that faces the others: h_s = mid_s edge_{s/32}
    __half lo[WC];     // (at most half an ulp of hi; its rounding leaves out at most 2^-25 of G's unit below 1024, 2^-36 of G above)
    float edge[4], whole;   // decay between the blocks' faces and where the chunk's state is; exp(G_C)
    __device__ __forceinline__ Sum2 sum(int t) const { return {hi[t], __half2float(lo[t])}; }
};

struct DecayBars {
    uint64_t full[8], empty[8], aux, beside, gfull[2], gfree[2];
    uint64_t s, p, y, scaled, out, ofree, staged, vl, dm0, dm, m, y2, m3, drain;
    uint32_t tmem;
    int gone;
};

template <int D, bool SUM, bool DOTS>
struct DecayLayout {
    static constexpr int HALVES = D / 64, PER = SUM ? 2 : 3;               // tiles per chunk
    static constexpr uint32_t HALF = WC * 128, TILE_BYTES = HALVES * HALF;  // tile: [half of D][128 steps][64 values]
    // Room for five tiles (six of 64 values), of which one is `beside`'s and, later in the chunk, out's.
    static constexpr int ROOM = D == 64 ? 6 : 5, SLOTS = DOTS ? ROOM - 1 : ROOM;
    // The order in which a chunk's tiles come, so that the slot that one takes is that of a tile
    // which is done with early enough: y after dM, x after Y (or, where out leaves from its place, after that), z after out.
    static constexpr int Y = 0, X = DOTS ? 1 : 2, Z = DOTS ? 2 : 1;
    static constexpr int GB = 2;                                            // chunks of gates
    static constexpr uint32_t M_HALF = D * 128, M_TERM = HALVES * M_HALF;   // M: [term][half of dk][dv rows][64]
    static constexpr uint32_t M_AT = ROOM * TILE_BYTES, GATES_AT = M_AT + 2 * M_TERM;
    static constexpr uint32_t BARS_AT = GATES_AT + GB * sizeof(WalkGates), NEED = BARS_AT + sizeof(DecayBars);
    static constexpr uint32_t BYTES = NEED > 117760 ? NEED : 117760;        // one CTA per SM: it takes all of the tensor memory
    static_assert(BYTES <= 232448, "227 KB of shared memory");
};

namespace decay_tmem {
constexpr uint32_t S = 0;     // x y^T (128), then P: each 16 columns give way to their two terms
constexpr uint32_t O = 128;   // x M, scaled, then out
constexpr uint32_t DM = 256;  // the chunk's part of M'^T
constexpr uint32_t VL = 384;  // terms of h z, 64 steps (3 x 32)
// Where only states are summed up, a place for each half of a chunk and two for dM.
constexpr uint32_t VL2 = S, DM2 = O;
}  // namespace decay_tmem

// A warpgroup's share of the registers: 640 x 96 at launch are 2 x 128 x 128 + 2 x 128 x 88 + 128 x 48.
template <bool MORE, int N>
__device__ __forceinline__ void set_registers() {
    if constexpr (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// tc_wait and tc_wait_warp (tensor_core.cuh) that sleep in the barrier for up to 0.1 ms at a time:
// polls read shared memory, which is what bounds this kernel.
__device__ __forceinline__ bool mbar_sleep(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(100000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool walk_wait(uint64_t *bar, uint32_t parity, volatile int *gone, const Control &ctl) {
    unsigned long long t0 = 0;
    while (!mbar_sleep(bar, parity)) {
        if (t0 == 0) {
            wait_for_last();   // (the limit is this kernel's own: what it waits for may in turn wait for the kernel before)
            t0 = global_timer_ns();
        }
        const unsigned long long now = global_timer_ns();
        if (*gone || now - t0 > ctl.timeout_ns) {
            *gone = 1;   // (recorded once, at the kernel's end: the code of each wait stays short)
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool walk_wait_warp(uint64_t *bar, uint32_t parity, volatile int *gone, const Control &ctl) {
    const bool ok = walk_wait(bar, parity, gone, ctl);
    __syncwarp();
    tc_fence_after();
    return ok;
}

// Four 8 x 8 matrices of bfloat16 (rows of 16 bytes, one address per lane), each transposed:
// lane t gets rows 2 (t % 4) and + 1 of column t / 4.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t at, uint32_t *v) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
}
// Sixteen tensor-memory lanes x 8 columns: lane t holds column t % 4 of rows t / 4 (a) and t / 4 + 8 (b), and column 4 + t % 4 (c, d).
__device__ __forceinline__ void tmem_st16x128b2(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Arrives on a barrier that counts warps.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

// One warp: the gates of a chunk from its log decays (four steps per lane, zeros past the end); returns their whole sum.
__device__ __forceinline__ Sum2 walk_gates(WalkGates &s, const float *raw, bool rev) {
    const int lane = threadIdx.x % 32;
    Sum2 in[4], run = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) in[i] = run = sum2_add(run, {clamp_gate(raw[i]), 0.f});
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const Sum2 other = {__shfl_up_sync(0xffffffffu, run.hi, o), __shfl_up_sync(0xffffffffu, run.lo, o)};
        if (lane >= o) run = sum2_add(other, run);
    }
    Sum2 before = {__shfl_up_sync(0xffffffffu, run.hi, 1), __shfl_up_sync(0xffffffffu, run.lo, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const Sum2 end = {__shfl_sync(0xffffffffu, run.hi, 31), __shfl_sync(0xffffffffu, run.lo, 31)};
    // Lanes 8b .. 8b+7 hold block b: its last sum, and the one before its first.
    const int edge = rev ? lane / 8 * 8 : lane / 8 * 8 + 7;
    const Sum2 face = {__shfl_sync(0xffffffffu, rev ? before.hi : run.hi, edge), __shfl_sync(0xffffffffu, rev ? before.lo : run.lo, edge)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Sum2 g = i < 3 ? sum2_add(before, in[i]) : run;
        s.hi[4 * lane + i] = g.hi, s.lo[4 * lane + i] = __float2half_rn(g.lo);
        s.mid[4 * lane + i] = rev ? decay(g, face) : decay(face, g);
    }
    if (lane % 8 == 0) s.edge[lane / 8] = rev ? decay(face, {0.f, 0.f}) : decay(end, face);
    if (lane == 31) s.whole = decay(end, {0.f, 0.f});
    return end;
}

// Sixteen values of a row, n of them exist (a multiple of 8).
__device__ __forceinline__ void store_row(__nv_bfloat16 *out, const uint32_t *r, int n) {
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
    if (n >= 8) *reinterpret_cast<uint4 *>(out) = make_uint4(p[0], p[1], p[2], p[3]);
    if (n >= 16) *reinterpret_cast<uint4 *>(out + 8) = make_uint4(p[4], p[5], p[6], p[7]);
}
__device__ __forceinline__ void store_row(float *out, const uint32_t *r, int n) {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
        if (i < n) *reinterpret_cast<uint4 *>(out + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
}

// SUM: the state that a segment adds up from zero, and its decay; no out.  dq and dk also make
// what d_g needs (dots, dump, cross).  Loops are kept rolled where registers allow, and kinds are
// kernels of their own: five roles share the instruction cache (unrolled, warps waited for
// instructions 3.6 times as long as they issued, and 8 x 4096 x 16 x 128 took 185 instead of 149
// us; with the kinds decided at run time and a record of errors inside each wait 130 instead of 113).
enum WalkKind { WALK_OUT, WALK_DQ, WALK_DK, WALK_DV, WALK_SUM, WALK_SUM_REV };

template <int D, WalkKind KIND>
__global__ void __launch_bounds__(kDecayThreads, 1) decay_walk_kernel(const __grid_constant__ DecayArgs a) {
    constexpr bool SUM = KIND == WALK_SUM || KIND == WALK_SUM_REV, rev = KIND == WALK_DK || KIND == WALK_DV || KIND == WALK_SUM_REV;
    constexpr bool dots = KIND == WALK_DQ || KIND == WALK_DK, dump = KIND == WALK_DQ, cross = KIND == WALK_DK;
    using L = DecayLayout<D, SUM, dots>;
    namespace tmem = decay_tmem;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t sm32 = smem_addr(sm);   // (1024-byte aligned: the kernel has no other shared memory)
    DecayBars &bar = *reinterpret_cast<DecayBars *>(sm + L::BARS_AT);
    WalkGates *gates = reinterpret_cast<WalkGates *>(sm + L::GATES_AT);
    volatile int *gone = &bar.gone;

    // Which walk: sequence, segment, head.
    const int segs = SUM ? a.segs - 1 : a.segs;
    const DecayRole &ro = a.role;
    unsigned id = blockIdx.x;
    const int head = id % a.Hv;
    id /= a.Hv;
    const int seg = id % segs + (SUM && rev ? 1 : 0);
    long long n = id / segs;
    if (!SUM && a.longest_first) {
        int *scratch = reinterpret_cast<int *>(sm);
        n = by_length<kDecayThreads>(a.offsets, a.N, a.S, (unsigned)n, scratch, scratch + kMostOrdered, reinterpret_cast<unsigned *>(scratch + 2 * kMostOrdered));
        fence_proxy_async_smem();   // (the tiles come there, by the async proxy, once all have read it)
        __syncthreads();
    }
    long long b = n, s0 = 0, len = a.S, slot0 = n * a.NC;
    if (a.offsets) {
        const Seq seq = seq_of(a.offsets, a.S, n);
        b = 0, s0 = seq.s0, len = seq.len, slot0 = s0 / WC + n;
    }
    if (a.segs > 1) {
        const long long off = seg * a.seg_chunks * WC, left = len > off ? len - off : 0, most = a.seg_chunks * WC;
        s0 += off, slot0 += seg * a.seg_chunks, len = left < most ? left : most;
    }
    const int chunks = __reduce_min_sync(0xffffffffu, (int)((len + WC - 1) / WC));   // (in a uniform register, as the loops over it then are)
    const size_t pair = (size_t)n * a.Hv + head, seg_at = pair * a.segs + seg;
    auto chunk_at = [&](int it) { return rev ? chunks - 1 - it : it; };   // the it-th chunk that the walk comes to
    const int wg = warp_uniform(threadIdx.x / 128), warp = warp_uniform(threadIdx.x / 32), tid = threadIdx.x % 128;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) mbar_init(&bar.full[i], 1), mbar_init(&bar.empty[i], 1);
        for (uint64_t *x : {&bar.aux, &bar.beside, &bar.gfull[0], &bar.gfull[1], &bar.s, &bar.y, &bar.y2, &bar.out, &bar.dm0, &bar.dm, &bar.drain}) mbar_init(x, 1);
        for (uint64_t *x : {&bar.p, &bar.scaled, &bar.ofree, &bar.staged, &bar.vl, &bar.m, &bar.m3}) mbar_init(x, 8);   // two warpgroups' warps
        mbar_init(&bar.gfree[0], 16), mbar_init(&bar.gfree[1], 16);
        *gone = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc_all(&bar.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = __reduce_min_sync(0xffffffffu, bar.tmem), tl = tm + ((uint32_t)(warp % 4 * 32) << 16);   // this warp's lanes
    constexpr int terms = 2;                // of M
    const bool third = dots && !a.gate16;   // and one more, in the first one's place once that has been multiplied
    bool ok = true;   // none of this thread's waits has run out
    auto tile = [&](int it, int which) { return L::PER * it + which; };   // the it-th chunk's; tile i is in slot i % SLOTS
    auto stage_at = [&](int it) { return dots ? (uint32_t)(L::ROOM - 1) * L::TILE_BYTES : (uint32_t)(tile(it, L::X) % L::SLOTS) * L::TILE_BYTES; };
    auto slot = [&](int i) { return (uint32_t)(i % L::SLOTS) * L::TILE_BYTES; };
    // Waits of the warps that issue: whole warps go on or stop together.
    auto all_wait = [&](uint64_t *x, uint32_t parity) {
        const bool there = __all_sync(0xffffffffu, walk_wait(x, parity, gone, a.ctl)) != 0;
        tc_fence_after();
        return there;
    };
    auto wait_tile = [&](int i) { return walk_wait_warp(&bar.full[i % L::SLOTS], (i / L::SLOTS) & 1, gone, a.ctl); };

    // Terms of h z, 32 of the chunk's steps 64h .. (the first half by `convert`, the second by `state`):
    // 16 steps at a time, transposed by the loads, so that a register holds two steps of value
    // row lane / 4 (+ 8, 16, 24), which is how the 16-lane stores to tensor memory want them.
    const bool rows = D == 128 || warp % 4 < 2;   // this warp's value rows exist
    auto values = [&](int it, int h) {
        uint64_t *there = SUM && h ? &bar.p : &bar.vl;
        if (!rows) {
            warp_arrive(there);
            return;
        }
        const int lane = threadIdx.x % 32, step0 = h * 64 + wg % 2 * 32, row0 = warp % 4 * 32 % D;
        uint32_t at = sm32 + slot(tile(it, L::Z)) + (uint32_t)(row0 / 64) * L::HALF + (uint32_t)(step0 + lane / 8 % 2 * 8 + lane % 8) * 128 +
                      (uint32_t)(((row0 % 64 / 8 + lane / 16) ^ (lane % 8)) << 4);
        const float *f = &gates[it % L::GB].mid[step0 + lane % 4 * 2], edge = gates[it % L::GB].edge[h * 2 + wg % 2] * (rev ? a.scale : 1.f);
        uint32_t to = tl + (SUM && h ? tmem::VL2 : tmem::VL) + wg % 2 * 16;
#pragma unroll 1
        for (int q = 0; q < 2; ++q, at += 16 * 128, f += 16, to += 8) {
            const float2 lo = mul2(*reinterpret_cast<const float2 *>(f), make_float2(edge, edge));        // h of steps 0 .. 7
            const float2 hi = mul2(*reinterpret_cast<const float2 *>(f + 8), make_float2(edge, edge));    // and 8 .. 15
#pragma unroll
            for (int x = 0; x < 2; ++x) {   // 16 value rows
                uint32_t v[4], t[4][3];
                ldmatrix4_trans(x ? at ^ 32 : at, v);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    split2<3>(mul2(make_float2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u)), i % 2 ? hi : lo), t[i]);
#pragma unroll
                for (int j = 0; j < 3; ++j) tmem_st16x128b2(to + (x << 20) + j * 32, t[0][j], t[2][j], t[1][j], t[3][j]);
            }
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(there);
    };

    let_next_start();
    if (wg < 2) {
        set_registers<true, 128>();
        wait_for_last();   // (the other roles touch the call's inputs and outputs, dots that nothing reads yet, and what waits by itself)
        // ------------------------------------------------------------------ state, out
        constexpr int HALF = D / 2;   // of dk: this thread's columns of M^T; of dv: its columns of out
        const int col0 = wg * HALF;
        const bool in = tid < ro.dv;
        const size_t outside = pair * ro.dk * ro.dv + (size_t)tid * ro.lane;
        float2 m[HALF / 2];
        float whole = 0.f;
#pragma unroll
        for (int i = 0; i < HALF / 2; ++i) m[i] = make_float2(0.f, 0.f);
        if (KIND == WALK_DV && a.segs > 1 && tid < D) {   // dk's states, whose rows are these columns
            const float *p = ro.seg_m + seg_at * D * D + state_at<D>(tid % HALF / 4, tid / HALF, col0) + tid % 4;
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
                const float v = p[4 * i];
                if (i % 2) m[i / 2].y = v;
                else m[i / 2].x = v;
            }
        } else if (!SUM && a.segs > 1 && tid < D) {
#pragma unroll
            for (int j = 0; j < HALF / 4; ++j) {
                const float4 v = *reinterpret_cast<const float4 *>(ro.seg_m + seg_at * D * D + state_at<D>(j, wg, tid));
                m[2 * j] = make_float2(v.x, v.y), m[2 * j + 1] = make_float2(v.z, v.w);
            }
        } else if (!SUM && ro.init && in) {
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
                const float v = col0 + i < ro.dk ? __ldg(ro.init + outside + (size_t)(col0 + i) * ro.col) : 0.f;
                if (i % 2) m[i / 2].y = v;
                else m[i / 2].x = v;
            }
        }
        // Terms of M: row tid of [term][half of dk][D rows][64].
        auto put_m = [&](int p, auto last) {   // columns 16p ..; `last`: the third term, in the first one's place
            constexpr bool LAST = decltype(last)::value;
            if (!rows) return;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int c = col0 + p * 16 + u * 8;
                const uint32_t at = sm32 + L::M_AT + (uint32_t)(c / 64) * L::M_HALF + swizzled(tid, c % 64 / 8);
                uint32_t t[4][3];
#pragma unroll
                for (int i = 0; i < 4; ++i) split2<LAST ? 3 : terms>(m[p * 8 + u * 4 + i], t[i]);
#pragma unroll
                for (int j = LAST ? 2 : 0; j < (LAST ? 3 : terms); ++j) {
                    const uint32_t v[4] = {t[0][j], t[1][j], t[2][j], t[3][j]};
                    st_shared16(at + (LAST ? 0 : j) * L::M_TERM, v);
                }
            }
        };
        auto give_m = [&] {   // M's terms are there
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&bar.m);
        };
        auto absorb = [&](uint32_t dm) {   // M' = exp(G_C) M + dM
            if (!rows) return;
#pragma unroll
            for (int p = 0; p < HALF / 16; p += 2) {
                uint32_t r[32];
                tmem_ld32(tl + dm + col0 + p * 16, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    m[p * 8 + i] = fma2(make_float2(whole, whole), m[p * 8 + i], make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
                if (!SUM) put_m(p, std::false_type()), put_m(p + 1, std::false_type());
                __syncwarp();
            }
        };
        if constexpr (SUM) {
            // A chunk's second half of h z is made before the last one's dM is read: the products always have something to do.
            float before = 0.f;
            auto last = [&](int it) {
                if (it > 0) {
                    whole = before;
                    absorb(it & 1 ? tmem::DM : tmem::DM2);
                    tc_fence_before();
                    warp_arrive(it & 1 ? &bar.m : &bar.scaled);
                }
            };
#pragma unroll 1
            for (int it = 0; it < chunks; ++it) {
                const int gb = it % L::GB;
                ok &= walk_wait(&bar.gfull[gb], (it / L::GB) & 1, gone, a.ctl);
                const float now = gates[gb].whole;
                __syncwarp();
                ok &= wait_tile(tile(it, L::Z));
                if (it > 0) ok &= walk_wait_warp(&bar.dm, (it - 1) & 1, gone, a.ctl);
                values(it, 1);
                warp_arrive(&bar.gfree[gb]);
                last(it);
                before = now;
            }
            if (chunks > 0) ok &= walk_wait_warp(&bar.dm, (chunks - 1) & 1, gone, a.ctl);
            last(chunks);
            if (tid < D)
#pragma unroll
                for (int j = 0; j < HALF / 4; ++j)
                    *reinterpret_cast<float4 *>(ro.seg_own + seg_at * D * D + state_at<D>(j, wg, tid)) = make_float4(m[2 * j].x, m[2 * j].y, m[2 * j + 1].x, m[2 * j + 1].y);
        } else {
#pragma unroll
            for (int p = 0; p < HALF / 16; ++p) put_m(p, std::false_type());
            // <other's state, M>, quarters of a thread's columns at a time, on their way while it waits
            // (all at once before the chunk's products are asked for: dk 204 us instead of 181, of two terms; behind h z's second half 221).
            constexpr int Q = HALF / 16;
            float4 theirs[2 * Q];
            float2 dot = make_float2(0.f, 0.f);
            auto fetch = [&](size_t kept, int quarter, int n) {
                if (tid < D)
#pragma unroll
                    for (int j = 0; j < n * Q; ++j) theirs[j] = *reinterpret_cast<const float4 *>(ro.other + kept + state_at<D>(quarter * Q + j, wg, tid));
            };
            auto multiply = [&](int quarter, int n) {
                if (tid < D)
#pragma unroll
                    for (int j = 0; j < n * Q; ++j) {
                        dot = fma2(m[2 * (quarter * Q + j)], make_float2(theirs[j].x, theirs[j].y), dot);
                        dot = fma2(m[2 * (quarter * Q + j) + 1], make_float2(theirs[j].z, theirs[j].w), dot);
                    }
            };
            give_m();
#pragma unroll 1
            for (int it = 0; it < chunks; ++it) {
                const int c = chunk_at(it), gb = it % L::GB;
                const long long t0 = (long long)c * WC;
                const WalkGates &gt = gates[gb];
                const int left = (int)min((long long)WC, len - t0);
                const size_t row = (size_t)(b * a.S + s0 + t0 + tid) * a.Hv + head;
                const size_t kept = ((size_t)(slot0 + c) * a.Hv + head) * D * D;
                if (cross) dot = make_float2(0.f, 0.f), fetch(kept, 0, 2);
                ok &= walk_wait(&bar.gfull[gb], (it / L::GB) & 1, gone, a.ctl);
                whole = gt.whole;
                __syncwarp();
                ok &= wait_tile(tile(it, L::Z));
                ok &= walk_wait_warp(&bar.dm0, it & 1, gone, a.ctl);
                if (cross) multiply(0, 2), fetch(kept, 2, 1);
                values(it, 1);
                warp_arrive(&bar.gfree[gb]);
                if (third) {
                    ok &= walk_wait_warp(&bar.y2, it & 1, gone, a.ctl);
#pragma unroll
                    for (int p = 0; p < HALF / 16; ++p) put_m(p, std::bool_constant<dots>());
                    fence_proxy_async_smem();
                    warp_arrive(&bar.m3);
                }
                if (cross) multiply(2, 1), fetch(kept, 3, 1);
                if (dump && tid < D)   // while Y and the rest of dM are made (175 us before them, 156 here)
#pragma unroll
                    for (int j = 0; j < HALF / 4; ++j)
                        *reinterpret_cast<float4 *>(ro.dump + kept + state_at<D>(j, wg, tid)) = make_float4(m[2 * j].x, m[2 * j].y, m[2 * j + 1].x, m[2 * j + 1].y);
                if (cross) {
                    multiply(3, 1);
                    float sum = (dot.x + dot.y) * whole;
                    __syncwarp();
#pragma unroll
                    for (int o = 16; o; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (tid % 32 == 0) ro.cross[((size_t)(slot0 + c) * a.Hv + head) * 8 + warp] = sum;
                }
                ok &= walk_wait_warp(&bar.dm, it & 1, gone, a.ctl);   // (behind Y, which reads M)
                if (third) ok &= walk_wait_warp(&bar.y, it & 1, gone, a.ctl);
                absorb(tmem::DM);
                give_m();
                ok &= walk_wait_warp(&bar.out, it & 1, gone, a.ctl);
                // Whole chunks leave by TMA, from x's place (dots: from `beside`'s), which is done with.
                if (ro.out32 || (a.offsets && left < WC)) {
#pragma unroll 1
                    for (int p = 0; p < HALF / 16; ++p) {
                        uint32_t r[16];
                        tmem_ld16(tl + tmem::O + col0 + p * 16, r);
                        tmem_wait_ld();
                        const size_t at = row * ro.dv + col0 + p * 16;
                        const int cols = tid < left ? ro.dv - col0 - p * 16 : 0;
                        if (ro.out32) store_row(static_cast<float *>(ro.out) + at, r, cols);
                        else store_row(static_cast<__nv_bfloat16 *>(ro.out) + at, r, cols);
                        __syncwarp();
                    }
                    tc_fence_before();
                    warp_arrive(&bar.ofree);
                } else {
                    const uint32_t stage = sm32 + stage_at(it);
#pragma unroll 1
                    for (int p = 0; p < HALF; p += 16) {
                        uint32_t r[16];
                        tmem_ld16(tl + tmem::O + col0 + p, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            uint32_t v[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) v[i] = pack_bf16(__uint_as_float(r[u * 8 + 2 * i]), __uint_as_float(r[u * 8 + 2 * i + 1]));
                            const int c = col0 + p + u * 8;
                            st_shared16(stage + (uint32_t)(c / 64) * L::HALF + swizzled(tid, c % 64 / 8), v);
                        }
                    }
                    tc_fence_before();
                    warp_arrive(&bar.ofree);
                    fence_proxy_async_smem();
                }
                warp_arrive(&bar.staged);
            }
            if (ro.fin && in && seg == (rev ? 0 : a.segs - 1)) {
#pragma unroll
                for (int i = 0; i < HALF; ++i)
                    if (col0 + i < ro.dk) ro.fin[outside + (size_t)(col0 + i) * ro.col] = i % 2 ? m[i / 2].y : m[i / 2].x;
            }
        }
        __syncwarp();
    } else if (wg < 4) {
        set_registers<false, 88>();
        // ------------------------------------------------------------------ convert
        constexpr int HALF = D / 2;   // columns of Y that this warpgroup scales
        const int part = wg - 2, rb = warp % 4;   // every other 32 columns of P; this warp's 32 rows
#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            const int gb = it % L::GB;
            const WalkGates &gt = gates[gb];
            ok &= walk_wait(&bar.gfull[gb], (it / L::GB) & 1, gone, a.ctl);
            ok &= wait_tile(tile(it, L::Z));
            if (it > 0) ok &= walk_wait_warp(SUM ? &bar.dm0 : &bar.dm, (it - 1) & 1, gone, a.ctl);   // the last half's terms are done with
            values(it, 0);
            if constexpr (!SUM) {
                const Sum2 mine = gt.sum(rb * 32 + threadIdx.x % 32);
                ok &= walk_wait_warp(&bar.s, it & 1, gone, a.ctl);
#pragma unroll 1
                for (int h = 0; h < 4; ++h) {   // 16 columns of P: every other block of 32, half of it at a time
                    const int cb = part + h / 2 * 2, c0 = cb * 32 + h % 2 * 16;
                    const uint32_t at = tl + tmem::S + c0;
                    uint32_t r[16];
                    if (rev ? cb < rb : cb > rb) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = 0;
                        tmem_st16(at, r);
                        continue;
                    }
                    tmem_ld16(at, r);
                    // D_ts = mid_s row, the second factor at most 1 off the diagonal; on it the other way
                    // round, as long as the block's decay is no more than 2^-60, else one exp2 a value.
                    const Sum2 face = rev ? cb ? gt.sum(cb * 32 - 1) : Sum2{0.f, 0.f} : gt.sum(cb * 32 + 31);
                    const bool diagonal = cb == rb;
                    const int t = threadIdx.x % 32 - h % 2 * 16;   // the diagonal's column
                    const float row = a.scale * (rev ? decay(face, mine) : decay(mine, face));
                    float2 w[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 o = *reinterpret_cast<const float4 *>(&gt.mid[c0 + 4 * i]);
                        w[2 * i] = mul2(make_float2(o.x, o.y), make_float2(row, row)), w[2 * i + 1] = mul2(make_float2(o.z, o.w), make_float2(row, row));
                    }
                    if (diagonal) {
                        if (fabsf(face.hi - gt.hi[cb * 32 + (rev ? 31 : 0)]) > 60.f) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float2 lo = __half22float2(*reinterpret_cast<const __half2 *>(&gt.lo[c0 + 2 * i])), hi = *reinterpret_cast<const float2 *>(&gt.hi[c0 + 2 * i]);
                                const float d0 = (mine.hi - hi.x) + (mine.lo - lo.x), d1 = (mine.hi - hi.y) + (mine.lo - lo.y);
                                w[i] = make_float2(a.scale * exp2_fast(fminf(rev ? -d0 : d0, 0.f)), a.scale * exp2_fast(fminf(rev ? -d1 : d1, 0.f)));
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (rev ? 2 * i < t : 2 * i > t) w[i].x = 0.f;
                            if (rev ? 2 * i + 1 < t : 2 * i + 1 > t) w[i].y = 0.f;
                        }
                    }
                    __syncwarp();
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = mul2(w[i], make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t t[2];
                        split2<2>(w[i], t);
                        r[i] = t[0], r[8 + i] = t[1];
                    }
                    tmem_st16(at, r);
                }
                // f Y in place, and its product with the row of `beside`.
                const float f = rev ? decay(gt.sum(WC - 1), mine) : a.scale * decay(mine, {0.f, 0.f});
                const int row = rb * 32 + threadIdx.x % 32;
                const unsigned char *be = sm + (L::ROOM - 1) * L::TILE_BYTES;
                if (dots) ok &= walk_wait_warp(&bar.beside, it & 1, gone, a.ctl);
                ok &= walk_wait_warp(&bar.y, it & 1, gone, a.ctl);
                float2 dot = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int c = part * HALF; c < part * HALF + HALF; c += 16) {
                    uint32_t r[16];
                    tmem_ld16(tl + tmem::O + c, r);
                    uint4 q[2];
                    if (dots)
#pragma unroll
                        for (int j = 0; j < 2; ++j) q[j] = *reinterpret_cast<const uint4 *>(be + c / 64 * L::HALF + swizzled(row, c % 64 / 8 + j));
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 y = mul2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), make_float2(f, f));
                        r[2 * i] = __float_as_uint(y.x), r[2 * i + 1] = __float_as_uint(y.y);
                        if (dots) {
                            const uint32_t w = i % 4 == 0 ? q[i / 4].x : i % 4 == 1 ? q[i / 4].y : i % 4 == 2 ? q[i / 4].z : q[i / 4].w;
                            dot = fma2(y, make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), dot);
                        }
                    }
                    tmem_st16(tl + tmem::O + c, r);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(&bar.scaled);
                if (dots) {
                    const long long t = (long long)chunk_at(it) * WC + row;
                    if (t < len) ro.dots[(size_t)part * a.B * a.S * a.Hv + (size_t)(b * a.S + s0 + t) * a.Hv + head] = dot.x + dot.y;
                    __syncwarp();
                }
            }
            warp_arrive(&bar.gfree[gb]);
        }
    } else {
        set_registers<false, 48>();
    if (warp == 16) {
        // ------------------------------------------------------------------ products
        const uint32_t id_s = mma_desc(128, 128), id_y = mma_desc(128, D), id_mn = mma_desc(128, D, false, true);
        auto tile_at = [&](int i) { return __reduce_min_sync(0xffffffffu, sm32 + slot(i)); };   // (uniform descriptors: tensor_core.cuh)
        auto all_tile = [&](int i) { return all_wait(&bar.full[i % L::SLOTS], (i / L::SLOTS) & 1); };
        auto scores = [&](int it) {   // S = x y^T
            ok &= all_tile(tile(it, L::Y));
            ok &= all_tile(tile(it, L::X));
            const uint64_t x = smem_desc(tile_at(tile(it, L::X)), 16, 1024), y = smem_desc(tile_at(tile(it, L::Y)), 16, 1024);
            if (elect_one() && ok) {
#pragma unroll 1
                for (int h = 0; h < L::HALVES; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_ss(tm + tmem::S, x + (h * L::HALF + k * 32 >> 4), y + (h * L::HALF + k * 32 >> 4), id_s, h > 0 || k > 0);
                mma_commit(&bar.s);
            }
            __syncwarp();
        };
        auto update = [&](int it, int h) {   // dM += (h z)^T y over 64 steps
            ok &= SUM ? all_wait(h ? &bar.p : &bar.vl, it & 1) : all_wait(&bar.vl, h);
            const uint32_t to = tm + (SUM && it % 2 ? tmem::DM2 : tmem::DM), from = tm + (SUM && h ? tmem::VL2 : tmem::VL);
            const uint64_t y = smem_desc(tile_at(tile(it, L::Y)) + h * 64 * 128, L::HALF, 1024);
            if (elect_one() && ok) {
#pragma unroll 1
                for (int j = 2; j >= 0; --j)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ts(to, from + j * 32 + k * 8, y + ((k * 2048) >> 4), id_mn, h > 0 || j < 2 || k > 0);
                mma_commit(h ? &bar.dm : &bar.dm0);
                if (h) mma_commit(&bar.empty[tile(it, L::Y) % L::SLOTS]);
                if (h && SUM) mma_commit(&bar.empty[tile(it, L::Z) % L::SLOTS]);
            }
            __syncwarp();
        };
        // What a chunk begins with: its scores and the first half of its dM (behind the last chunk's out).
        auto begin = [&](int it) {
            if constexpr (!SUM) {
                scores(it);
                ok &= all_wait(&bar.m, it & 1);   // dM has been read (and M's terms are there)
            } else {
                ok &= all_tile(tile(it, L::Y));
                if (it > 1) ok &= all_wait(it % 2 ? &bar.scaled : &bar.m, (it / 2 - 1) & 1);   // this dM has been read
            }
            update(it, 0);
        };
#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            begin(it);
            if constexpr (!SUM) {   // Y = x M
                if (it > 0) ok &= all_wait(&bar.ofree, (it - 1) & 1);
                const uint64_t x = smem_desc(tile_at(tile(it, L::X)), 16, 1024), y = smem_desc(__reduce_min_sync(0xffffffffu, sm32 + L::M_AT), 16, 1024);
                if (elect_one() && ok) {
#pragma unroll 1
                    for (int j = terms - 1; j >= 0; --j)   // the small term first
#pragma unroll 1
                        for (int h = 0; h < L::HALVES; ++h)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_ss(tm + tmem::O, x + (h * L::HALF + k * 32 >> 4), y + (j * L::M_TERM + h * L::M_HALF + k * 32 >> 4), id_y, j < terms - 1 || h > 0 || k > 0);
                    mma_commit(third ? &bar.y2 : &bar.y);
                    if (dots && !third) mma_commit(&bar.empty[tile(it, L::X) % L::SLOTS]);
                }
                __syncwarp();
            }
            update(it, 1);
            if (third) {
                ok &= all_wait(&bar.m3, it & 1);
                const uint64_t x = smem_desc(tile_at(tile(it, L::X)), 16, 1024), y = smem_desc(__reduce_min_sync(0xffffffffu, sm32 + L::M_AT), 16, 1024);
                if (elect_one() && ok) {
#pragma unroll 1
                    for (int h = 0; h < L::HALVES; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k) mma_ss(tm + tmem::O, x + (h * L::HALF + k * 32 >> 4), y + (h * L::M_HALF + k * 32 >> 4), id_y, true);
                    mma_commit(&bar.y);
                    mma_commit(&bar.empty[tile(it, L::X) % L::SLOTS]);
                }
                __syncwarp();
            }
            if constexpr (!SUM) {   // out = f Y + P z
                ok &= all_wait(&bar.scaled, it & 1);   // (and P, made before; z has been read for h z)
                const uint64_t z = smem_desc(tile_at(tile(it, L::Z)), L::HALF, 1024);
                if (elect_one() && ok) {
#pragma unroll 1
                    for (int j = 1; j >= 0; --j)   // the small term first
#pragma unroll
                        for (int k = 0; k < 8; ++k) mma_ts(tm + tmem::O, tm + tmem::S + k * 16 + j * 8, z + (k * 2048 >> 4), id_mn, true);
                    mma_commit(&bar.out);
                    mma_commit(&bar.empty[tile(it, L::Z) % L::SLOTS]);
                }
                __syncwarp();
            }
        }
        if (elect_one() && (!ok || *gone)) drain_products(&bar.drain, a.ctl);
        __syncwarp();
    } else if (warp == 17) {
        // ------------------------------------------------------------------ copies
        // (Only in a packed batch a walk's last rows may be another sequence's; past S, TMA fills with zeros.)
        int aux = 0, sent = 0;
        const int tiles = L::PER * chunks;
#pragma unroll 1
        for (int i = 0; i < tiles && ok; ++i) {
            const int it = i / L::PER, which = i % L::PER, sl = i % L::SLOTS;
            ok &= all_wait(&bar.empty[sl], ((i / L::SLOTS) & 1) ^ 1);
            if (!ok) break;
            const long long t0 = (long long)chunk_at(it) * WC;
            const int left = (int)min((long long)WC, len - t0);
            const bool clear = a.offsets && which != L::X && left < WC;   // rows of y and z past the end count as zero
            unsigned char *dst = sm + slot(i);
            if (elect_one()) {
                const CUtensorMap *map = which == L::X ? &ro.x : which == L::Y ? &ro.y : &ro.z;
                const int h = head / (which == L::X ? ro.gx : which == L::Y ? ro.gy : ro.gz), s = (int)(s0 + t0);
                uint64_t *on = clear ? &bar.aux : &bar.full[sl];
                // (The test hook makes CTA `stall_tile` expect 16 bytes that never come.)
                mbar_arrive_expect_tx(on, L::TILE_BYTES + ((int)blockIdx.x == a.ctl.stall_tile ? 16 : 0));
#pragma unroll
                for (int x = 0; x < L::HALVES; ++x) {
                    tma_load_4d(dst + x * L::HALF, map, x * 64, h, s, (int)b, on);
                    tma_load_4d(dst + x * L::HALF + 8192, map, x * 64, h, s + 64, (int)b, on);
                }
                if (it + 1 < chunks) {   // and the next chunk's tile into L2
                    const int s1 = (int)(s0 + (long long)chunk_at(it + 1) * WC);
#pragma unroll
                    for (int x = 0; x < L::HALVES; ++x) {
                        tma_prefetch_4d(map, x * 64, h, s1, (int)b);
                        tma_prefetch_4d(map, x * 64, h, s1 + 64, (int)b);
                    }
                }
            }
            __syncwarp();
            sent = i + 1;
            if (clear) {
                ok &= all_wait(&bar.aux, aux++ & 1);
                const uint32_t z[4] = {0, 0, 0, 0};
                for (int k = threadIdx.x % 32; k < (WC - left) * 8; k += 32)
#pragma unroll
                    for (int x = 0; x < L::HALVES; ++x) st_shared16(sm32 + slot(i) + x * L::HALF + (left + k / 8) * 128 + k % 8 * 16, z);
                fence_proxy_async_smem();
                __syncwarp();
                if (elect_one() && ok) mbar_arrive(&bar.full[sl]);
                __syncwarp();
            }
        }
        if (elect_one() && (!ok || *gone)) {   // copies still in flight
            for (int i = max(0, sent - L::SLOTS); i < sent; ++i) drain_wait(&bar.full[i % L::SLOTS], (i / L::SLOTS) & 1, a.ctl);
            if (aux) drain_wait(&bar.aux, (aux - 1) & 1, a.ctl);
        }
        __syncwarp();
    } else if (warp == 18) {
        // ------------------------------------------------------------------ gates
        const int lane = threadIdx.x % 32;
        float raw[4];
        Sum2 all = {0.f, 0.f};
        auto read = [&](int it) {
            const long long t0 = (long long)chunk_at(it) * WC + 4 * lane, row = (b * a.S + s0 + t0) * a.Hv + head;
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[i] = t0 + i < len ? load_any(a.g, a.gate16, row + (long long)i * a.Hv) : 0.f;
        };
        // (A sum's chunks are short, and dk loads states besides: 1 x 131072 x 16 x 64 forward 409 -> 384 us, dk
        // at 8 x 4096 x 16 x 128 181 -> 172, of two terms.  For the others it is more code: dq 162 -> 165.)
        constexpr bool far = SUM || cross;
        auto ahead = [&](int it) {   // into L2
            const long long t0 = (long long)chunk_at(it) * WC + 4 * lane, row = (b * a.S + s0 + t0) * a.Hv + head;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t0 + i < len) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(a.g) + (row + (long long)i * a.Hv) * (a.gate16 ? 2 : 4)));
        };
        if (chunks > 0) read(0);
        if (far)
            for (int it = 1; it < min(chunks, 3); ++it) ahead(it);
#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            const int gb = it % L::GB;
            ok &= all_wait(&bar.gfree[gb], ((it / L::GB) & 1) ^ 1);
            const Sum2 end = walk_gates(gates[gb], raw, rev);
            if (SUM) all = sum2_add(all, end);
            __syncwarp();
            warp_arrive(&bar.gfull[gb]);
            if (it + 1 < chunks) {
                read(it + 1);
                if (far && it + 3 < chunks) ahead(it + 3);
                if (cross && lane == 0)   // and the states that the next chunk's are compared with, into L2
                    bulk_prefetch(ro.other + ((size_t)(slot0 + chunk_at(it + 1)) * a.Hv + head) * D * D, D * D * 4);
            }
        }
        if (SUM) {
            wait_for_last();   // (the join of the walk before may not have read its own yet)
            if (lane == 0) ro.seg_decay[seg_at] = decay(all, {0.f, 0.f});
        }
    } else if (!SUM) {
        // ------------------------------------------------------------------ out to memory
        bool some = false;
        int asked = 0;   // tiles of `beside`
        auto beside = [&](int it) {
            if (!dots || it >= chunks || !ok) return;
            if (elect_one()) {
                const int s = (int)(s0 + (long long)chunk_at(it) * WC), h = head / ro.gb;
                unsigned char *dst = sm + (L::ROOM - 1) * L::TILE_BYTES;
                mbar_arrive_expect_tx(&bar.beside, L::TILE_BYTES);
#pragma unroll
                for (int x = 0; x < L::HALVES; ++x) {
                    tma_load_4d(dst + x * L::HALF, &ro.b, x * 64, h, s, (int)b, &bar.beside);
                    tma_load_4d(dst + x * L::HALF + 8192, &ro.b, x * 64, h, s + 64, (int)b, &bar.beside);
                }
            }
            __syncwarp();
            asked = it + 1;
        };
        beside(0);
#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            ok &= all_wait(&bar.staged, it & 1);
            const long long t0 = (long long)chunk_at(it) * WC;
            const int left = (int)min((long long)WC, len - t0);
            const bool staged = !ro.out32 && !(a.offsets && left < WC);
            if (elect_one() && ok) {
                if (staged) {
                    const unsigned char *src = sm + stage_at(it);
#pragma unroll
                    for (int x = 0; x < 2 * L::HALVES; ++x)
                        if (x / 2 * 64 < ro.dv && (x % 2 == 0 || left > 64))
                            tma_store_4d(&ro.o, src + x / 2 * L::HALF + x % 2 * 8192, x / 2 * 64, head, (int)(s0 + t0) + x % 2 * 64, (int)b);
                    bulk_commit_group();
                    bulk_wait_group_read<0>();
                    some = true;
                }
                if (!dots) mbar_arrive(&bar.empty[tile(it, L::X) % L::SLOTS]);
            }
            __syncwarp();
            beside(it + 1);
        }
        if (dots && elect_one() && (!ok || *gone) && asked) drain_wait(&bar.beside, (asked - 1) & 1, a.ctl);
        __syncwarp();
        if (some) bulk_wait_group_all();
        __syncwarp();
    }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free_all(tm);
    if (threadIdx.x == 0 && *gone) record_error(a.ctl.hdr, (int)blockIdx.x);
}

// The state that enters each segment, from the state that enters the first in walking order:
// m' = decay m + own.  A thread per four values of a (role, sequence, head).
template <int D, bool REV>
__global__ void __launch_bounds__(256) decay_join_kernel(const __grid_constant__ DecayArgs a) {
    const DecayRole &ro = a.role;
    const size_t pair = blockIdx.y;
    let_next_start();
    wait_for_last();
    const int i = blockIdx.x * 256 + threadIdx.x, j4 = i / (2 * D), wg = i / D % 2, dv = i % D;   // as state_at
    float4 m = q_zero();
    if (ro.init && dv < ro.dv) {
        const float *p = ro.init + pair * ro.dk * ro.dv + (size_t)dv * ro.lane;
        float *f = &m.x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = wg * (D / 2) + j4 * 4 + k;
            f[k] = c < ro.dk ? __ldg(p + (size_t)c * ro.col) : 0.f;
        }
    }
    float *enter = const_cast<float *>(ro.seg_m);
    constexpr int AHEAD = 8;   // sums on their way at a time
    for (int s0 = 0; s0 < a.segs; s0 += AHEAD) {
        float4 own[AHEAD];
        float d[AHEAD];
        auto at = [&](int k) { return pair * a.segs + (REV ? a.segs - 1 - (s0 + k) : s0 + k); };
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (s0 + k + 1 < a.segs) own[k] = *reinterpret_cast<const float4 *>(ro.seg_own + at(k) * D * D + (size_t)i * 4), d[k] = ro.seg_decay[at(k)];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (s0 + k < a.segs) {
                *reinterpret_cast<float4 *>(enter + at(k) * D * D + (size_t)i * 4) = m;
                m = make_float4(fmaf(d[k], m.x, own[k].x), fmaf(d[k], m.y, own[k].y), fmaf(d[k], m.z, own[k].z), fmaf(d[k], m.w, own[k].w));
            }
    }
}

}  // namespace qs
