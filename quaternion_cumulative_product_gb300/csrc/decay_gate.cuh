// decay_gate.cuh -- gradient of the log decays of linear attention, bfloat16.
//
// dg_u holds what crosses step u, from a state or key before it to a query or state from it on:
//
//     dg_u = sum_{t>=u>s} Z_ts + sum_{t>=u} a_t + sum_{s<u} b_s + exp(G_C) <M, dM'>
//     Z_ts = scale D_ts <q_t, k_s> <do_t, v_s>          (s < t, both in the chunk)
//     a_t  = scale exp(G_t) <q_t, M do_t>,   b_s = exp(G_C - G_s) <k_s, dM' v_s>
//
// with the states M and dM' that enter the chunk from either side.  a, b and the last term come
// from the walks (decay_walk.cuh: dots, cross).  Each term has the factor exp(g_u), and no two
// of them cancel (sums of <q, dq> - <k, dk> from a step on would: delta_common.cuh).
//
// One CTA per (chunk, head), two on an SM.  Q K^T and dO V^T on the tensor cores (products of
// bfloat16 values, exact up to fp32's sums), rows t in tensor-memory lanes.  A warp takes 32 x 32
// pieces of Z: prefix sums along its rows, sums down the columns by exchanges that halve the columns
// a lane still holds; sums of whole rows carry over to the pieces on the right.
//
// Bound: memory (the four tensors once more) and the latency of a CTA's steps: 142 us at
// 8 x 4096 x 16 x 128, 537 MB, 3.8 TB/s (180 us with eight warps instead of sixteen and without the
// next CTA's tiles in L2).
#pragma once

#include "decay_walk.cuh"

namespace qs {

constexpr int kGateThreads = 512;

struct GateArgs {
    CUtensorMap q, k, v, o;       // o: dO
    const void *g;
    void *dg;
    const float *a, *b, *cross;   // [2][B, S, Hv], the same, [slots, Hv, 8]
    const int *offsets;
    long long B, S, N, NC, slots;
    int Hv, shared;               // value heads that share a key head
    unsigned ahead;               // CTAs that run at once
    bool gate16;
    float scale;
    Control ctl;
};

struct GateShared {
    WalkGates gates;
    float columns[4][WC];     // [rows' block][u] sums of the rows' prefixes
    float rows[4][WC];        // [columns' block][t] sums of a row's pieces
    float suma[4], sumb[4];
    uint64_t q, k, v, o, s, e, drain;
    uint32_t tmem;
    int gone;
};

template <int D>
struct GateLayout {
    static constexpr int HALVES = D / 64;
    static constexpr uint32_t HALF = WC * 128, TILE_BYTES = HALVES * HALF, AT = 3 * TILE_BYTES;
    static constexpr uint32_t BYTES = AT + sizeof(GateShared);   // two CTAs per SM, 256 columns of tensor memory each
    static_assert(2 * (BYTES + 1024) <= 233472, "two CTAs per SM");
};

template <int D>
__global__ void __launch_bounds__(kGateThreads, 2) decay_gate_kernel(const __grid_constant__ GateArgs a) {
    using L = GateLayout<D>;
    extern __shared__ __align__(1024) unsigned char sm[];
    GateShared &sh = *reinterpret_cast<GateShared *>(sm + L::AT);
    volatile int *gone = &sh.gone;
    const uint32_t sm32 = smem_addr(sm);
    const int head = blockIdx.x % a.Hv, warp = warp_uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const long long slot = blockIdx.x / a.Hv;
    long long b, s0, len, c;
    if (a.offsets) {
        long long lo = 0, hi = a.N;   // the last n whose first slot is not past this one
        while (hi - lo > 1) {
            const long long mid = (lo + hi) / 2;
            if (seq_of(a.offsets, a.S, mid).s0 / WC + mid <= slot) lo = mid;
            else hi = mid;
        }
        const Seq seq = seq_of(a.offsets, a.S, lo);
        b = 0, s0 = seq.s0, len = seq.len, c = slot - (seq.s0 / WC + lo);
    } else {
        b = slot / a.NC, s0 = 0, len = a.S, c = slot % a.NC;
    }
    const long long t0 = c * WC;
    if (c < 0 || t0 >= len) {   // (a slot that holds no chunk; what comes after this kernel takes its end for that of the walks, too)
        wait_for_last();
        return;
    }
    const int left = (int)min((long long)WC, len - t0);
    const size_t row0 = (size_t)(b * a.S + s0 + t0) * a.Hv + head;

    // What the walks have left, for the last step's warps (step u = warp * 32 + lane); on its way meanwhile.
    float fa = 0.f, fb = 0.f, whole = 0.f;
    let_next_start();
    if (warp < 4) {
        wait_for_last();
        const size_t half = (size_t)a.B * a.S * a.Hv, at = row0 + (size_t)(warp * 32 + lane) * a.Hv;
        if (warp * 32 + lane < left) fa = a.a[at] + a.a[half + at], fb = a.b[at] + a.b[half + at];
        if (lane < 8) whole = a.cross[((size_t)slot * a.Hv + head) * 8 + lane];
    }
    if (threadIdx.x == 32) {
        for (uint64_t *x : {&sh.q, &sh.k, &sh.v, &sh.o, &sh.s, &sh.e, &sh.drain}) mbar_init(x, 1);
        *gone = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_addr(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = (uint32_t)warp_uniform((int)sh.tmem), tl = tm + ((uint32_t)(warp % 4 * 32) << 16);
    bool ok = true;
    if (warp == 12) {   // products (a warp without a piece of Z, as the gates' one): Q, K and V come first, dO in Q's place once S is made
        auto load = [&](const CUtensorMap *map, int at, int h, uint64_t *on) {
            mbar_arrive_expect_tx(on, L::TILE_BYTES);
#pragma unroll
            for (int x = 0; x < L::HALVES; ++x) {
                tma_load_4d(sm + at * L::TILE_BYTES + x * L::HALF, map, x * 64, h, (int)(s0 + t0), (int)b, on);
                tma_load_4d(sm + at * L::TILE_BYTES + x * L::HALF + 8192, map, x * 64, h, (int)(s0 + t0) + 64, (int)b, on);
            }
        };
        auto product = [&](uint32_t d, int x, int y, uint64_t *done) {
            const uint64_t p = smem_desc(sm32 + x * L::TILE_BYTES, 16, 1024), q = smem_desc(sm32 + y * L::TILE_BYTES, 16, 1024);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t at = ((k / 4) * L::HALF + (k % 4) * 32) >> 4;
                mma_ss(tm + d, p + at, q + at, mma_desc(128, 128), k > 0);
            }
            mma_commit(done);
        };
        const int kh = head / a.shared;
        if (elect_one()) {
            load(&a.q, 0, kh, &sh.q), load(&a.k, 1, kh, &sh.k), load(&a.v, 2, head, &sh.v);
#pragma unroll
            for (int x = 0; x < 2 * L::HALVES; ++x) tma_prefetch_4d(&a.o, x / 2 * 64, head, (int)(s0 + t0) + x % 2 * 64, (int)b);
            // The CTA that likely comes next on this SM: its tiles into L2 meanwhile.
            const unsigned next = blockIdx.x + a.ahead;
            if (!a.offsets && next < gridDim.x) {
                const int h = next % a.Hv, s = (int)(next / a.Hv % a.NC) * WC, nb = (int)(next / a.Hv / a.NC);
#pragma unroll
                for (int x = 0; x < 2 * L::HALVES; ++x) {
                    tma_prefetch_4d(&a.q, x / 2 * 64, h / a.shared, s + x % 2 * 64, nb);
                    tma_prefetch_4d(&a.k, x / 2 * 64, h / a.shared, s + x % 2 * 64, nb);
                    tma_prefetch_4d(&a.v, x / 2 * 64, h, s + x % 2 * 64, nb);
                }
            }
        }
        __syncwarp();
        auto both = [&](uint64_t *x) { ok &= __all_sync(0xffffffffu, tc_wait_warp(x, 0, gone, a.ctl)) != 0; };
        both(&sh.q), both(&sh.k);
        if (elect_one() && ok) product(0, 0, 1, &sh.s);
        __syncwarp();
        both(&sh.s);
        bool sent = false;
        if (elect_one() && ok) load(&a.o, 0, head, &sh.o), sent = true;
        __syncwarp();
        both(&sh.v), both(&sh.o);
        if (elect_one() && ok) product(128, 0, 2, &sh.e);
        __syncwarp();
        if (elect_one() && (!ok || *gone)) {
            for (uint64_t *x : {&sh.q, &sh.k, &sh.v}) drain_wait(x, 0, a.ctl);
            if (sent) drain_wait(&sh.o, 0, a.ctl);
            drain_products(&sh.drain, a.ctl);
        }
        __syncwarp();
    }
    if (warp == 8) {
        float raw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = 4 * lane + i < left ? load_any(a.g, a.gate16, row0 + (size_t)(4 * lane + i) * a.Hv) : 0.f;
        walk_gates(sh.gates, raw, false);
    }
    for (int i = threadIdx.x; i < 4 * WC; i += kGateThreads) (&sh.rows[0][0])[i] = (&sh.columns[0][0])[i] = 0.f;
    __syncthreads();
    ok &= tc_wait_warp(&sh.s, 0, gone, a.ctl);
    ok &= tc_wait_warp(&sh.e, 0, gone, a.ctl);
    const WalkGates &gt = sh.gates;
    const int rb = warp % 4, t = rb * 32 + lane;
    const Sum2 mine = gt.sum(t);
    const bool live = t < left;
    const int cb = warp / 4;
    if (cb <= rb) {
        const bool diagonal = cb == rb;
        const float row = diagonal ? 0.f : a.scale * decay(mine, gt.sum(cb * 32 + 31));
        float z[32], sum = 0.f;
#pragma unroll
        for (int p = 0; p < 32; p += 16) {
            uint32_t r[16], e[16];
            tmem_ld16(tl + cb * 32 + p, r);
            tmem_ld16(tl + 128 + cb * 32 + p, e);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float w;
                if (diagonal) w = a.scale * exp2_fast(p + i < lane ? (mine.hi - gt.hi[cb * 32 + p + i]) + (mine.lo - __half2float(gt.lo[cb * 32 + p + i])) : 0.f);
                else w = row * gt.mid[cb * 32 + p + i];
                const bool on = live && (!diagonal || p + i < lane);
                const float x = on ? w * __uint_as_float(r[i]) * __uint_as_float(e[i]) : 0.f;
                z[p + i] = !diagonal || p + i <= lane ? sum : 0.f;   // what the row holds before this column
                sum += x;
            }
        }
        sh.rows[cb][t] = sum;
        // The warp's 32 rows: each exchange halves the columns that a lane still holds.
#pragma unroll
        for (int k = 0; k < 5; ++k)
#pragma unroll
            for (int j = 0; j < 16 >> k; ++j) {
                const int n = 16 >> k;
                const bool up = lane & n;
                const float give = up ? z[j] : z[j + n], keep = up ? z[j + n] : z[j];
                z[j] = keep + __shfl_xor_sync(0xffffffffu, give, n);
            }
        sh.columns[rb][cb * 32 + lane] = z[0];   // (lane's bits chose column `lane`)
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tm) : "memory");
    if (warp >= 4) return;
    // A warp takes the 32 steps u of block `warp`.
    const int u = warp * 32 + lane;
    float d = 0.f, below = 0.f, here = 0.f;
    for (int r = warp; r < 4; ++r) d += sh.columns[r][u];
    // Rows' sums over the blocks before this one: of the rows below, whole; of its own, from step u on.
    for (int cb = 0; cb < warp; ++cb) {
        here += sh.rows[cb][u];
        for (int r = warp + 1; r < 4; ++r) below += sh.rows[cb][r * 32 + lane];
    }
    float from = fa + here, upto = fb, sa = fa, sb = fb;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const float right = __shfl_down_sync(0xffffffffu, from, o), earlier = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane + o < 32) from += right;
        if (lane >= o) upto += earlier;
        below += __shfl_xor_sync(0xffffffffu, below, o);
        whole += __shfl_xor_sync(0xffffffffu, whole, o);
        sa += __shfl_xor_sync(0xffffffffu, sa, o);
        sb += __shfl_xor_sync(0xffffffffu, sb, o);
    }
    if (lane == 0) sh.suma[warp] = sa, sh.sumb[warp] = sb;
    named_bar_sync(1, 128);
    float before = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane == 0) before = 0.f;
    for (int r = 0; r < warp; ++r) before += sh.sumb[r];
    for (int r = warp + 1; r < 4; ++r) from += sh.suma[r];
    if (u < left) store_any(a.dg, a.gate16, row0 + (size_t)u * a.Hv, d + below + from + before + whole);
}

}  // namespace qs
