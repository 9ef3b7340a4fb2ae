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
// Persistent CTAs, two on an SM, a (chunk, head) at a time.  Q K^T and dO V^T on the tensor cores
// (products of bfloat16 values, exact up to fp32's sums), rows t in tensor-memory lanes.  A warp takes
// 32 x 32 pieces of Z: prefix sums along its rows, sums down the columns by exchanges that halve the
// columns a lane still holds; sums of whole rows carry over to the pieces on the right.  The next
// chunk's tiles come in meanwhile.
//
// Bound: memory (the four tensors once more) and the latency of a chunk's steps: 120 us at
// 8 x 4096 x 16 x 128, 537 MB, 4.5 TB/s (a CTA for each chunk 142 us; with eight warps instead of
// sixteen and without the next CTA's tiles in L2 180).
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
    bool gate16;
    float scale;
    Control ctl;
};

struct GateShared {
    // (two chunks' of each: the last step of one goes on while the next is begun)
    WalkGates gates[2];
    float columns[2][4][WC];  // [rows' block][u] sums of the rows' prefixes (read from the diagonal on)
    float rows[2][4][WC];     // [columns' block][t] sums of a row's pieces (up to it)
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

// Where a unit's chunk is: unit = slot * Hv + head.
struct GateUnit {
    long long unit, slot, b, s, row0;   // row0: of [B, S, Hv]
    int head, left;                     // steps of the chunk
};

// The first unit from `unit` on, in strides of the grid, that holds a chunk; past the last: false.
__device__ __forceinline__ bool gate_unit(const GateArgs &a, long long unit, GateUnit *u) {
    for (; unit < a.slots * a.Hv; unit += gridDim.x) {
        const long long slot = unit / a.Hv;
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
        if (c < 0 || t0 >= len) continue;   // (a slot that holds no chunk)
        u->unit = unit, u->slot = slot, u->b = b, u->s = s0 + t0, u->head = (int)(unit % a.Hv);
        u->left = (int)min((long long)WC, len - t0), u->row0 = (b * a.S + s0 + t0) * a.Hv + u->head;
        return true;
    }
    return false;
}

template <int D>
__global__ void __launch_bounds__(kGateThreads, 2) decay_gate_kernel(const __grid_constant__ GateArgs a) {
    using L = GateLayout<D>;
    extern __shared__ __align__(1024) unsigned char sm[];
    GateShared &sh = *reinterpret_cast<GateShared *>(sm + L::AT);
    volatile int *gone = &sh.gone;
    const uint32_t sm32 = smem_addr(sm);
    const int warp = warp_uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    GateUnit u;
    let_next_start();
    if (!gate_unit(a, blockIdx.x, &u)) {   // (what comes after this kernel takes its end for that of the walks, too)
        wait_for_last();
        return;
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
    if (warp < 4) wait_for_last();   // (they read what the walks have left)
    const uint32_t tm = (uint32_t)warp_uniform((int)sh.tmem), tl = tm + ((uint32_t)(warp % 4 * 32) << 16);
    bool ok = true;
    int loaded = 0, sent = 0;   // warp 12: chunks whose Q, K and V, whose dO have been asked for
    auto load = [&](const CUtensorMap *map, int at, const GateUnit &g, int h, uint64_t *on) {
        mbar_arrive_expect_tx(on, L::TILE_BYTES);
#pragma unroll
        for (int x = 0; x < L::HALVES; ++x) {
            tma_load_4d(sm + at * L::TILE_BYTES + x * L::HALF, map, x * 64, h, (int)g.s, (int)g.b, on);
            tma_load_4d(sm + at * L::TILE_BYTES + x * L::HALF + 8192, map, x * 64, h, (int)g.s + 64, (int)g.b, on);
        }
    };
    auto begin = [&](const GateUnit &g) {   // Q, K and V come first, dO in Q's place once S is made
        if (elect_one()) {
            load(&a.q, 0, g, g.head / a.shared, &sh.q), load(&a.k, 1, g, g.head / a.shared, &sh.k), load(&a.v, 2, g, g.head, &sh.v);
#pragma unroll
            for (int x = 0; x < 2 * L::HALVES; ++x) tma_prefetch_4d(&a.o, x / 2 * 64, g.head, (int)g.s + x % 2 * 64, (int)g.b);
        }
        __syncwarp();
        ++loaded;
    };
    if (warp == 12) begin(u);
    bool more = true;
#pragma unroll 1
    for (int n = 0; more; ++n) {
        const WalkGates &gt = sh.gates[n & 1];
        float(*columns)[WC] = sh.columns[n & 1], (*rows)[WC] = sh.rows[n & 1];
        // What the walks have left, for the last step's warps (step warp * 32 + lane); on its way meanwhile.
        float fa = 0.f, fb = 0.f, whole = 0.f;
        if (warp < 4) {
            const size_t half = (size_t)a.B * a.S * a.Hv, at = u.row0 + (size_t)(warp * 32 + lane) * a.Hv;
            if (warp * 32 + lane < u.left) fa = a.a[at] + a.a[half + at], fb = a.b[at] + a.b[half + at];
            if (lane < 8) whole = a.cross[((size_t)u.slot * a.Hv + u.head) * 8 + lane];
        }
        if (warp == 8) {
            float raw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[i] = 4 * lane + i < u.left ? load_any(a.g, a.gate16, u.row0 + (size_t)(4 * lane + i) * a.Hv) : 0.f;
            walk_gates(sh.gates[n & 1], raw, false);
        }
        if (warp == 12) {   // products (a warp without a piece of Z, as the gates' one)
            auto product = [&](uint32_t d, int x, int y, uint64_t *done) {
                const uint64_t p = smem_desc(sm32 + x * L::TILE_BYTES, 16, 1024), q = smem_desc(sm32 + y * L::TILE_BYTES, 16, 1024);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t at = ((k / 4) * L::HALF + (k % 4) * 32) >> 4;
                    mma_ss(tm + d, p + at, q + at, mma_desc(128, 128), k > 0);
                }
                mma_commit(done);
            };
            auto both = [&](uint64_t *x) { ok &= __all_sync(0xffffffffu, tc_wait_warp(x, n & 1, gone, a.ctl)) != 0; };
            both(&sh.q), both(&sh.k);
            if (elect_one() && ok) product(0, 0, 1, &sh.s);
            __syncwarp();
            both(&sh.s);
            if (ok) {
                if (elect_one()) load(&a.o, 0, u, u.head, &sh.o);
                __syncwarp();
                ++sent;
            }
            both(&sh.v), both(&sh.o);
            if (elect_one() && ok) product(128, 0, 2, &sh.e);
            __syncwarp();
        }
        __syncthreads();
        ok &= tc_wait_warp(&sh.s, n & 1, gone, a.ctl);
        ok &= tc_wait_warp(&sh.e, n & 1, gone, a.ctl);
        if (warp == 12) {   // the next chunk's tiles, while the others work on this one's products
            ok = __all_sync(0xffffffffu, ok) != 0;
            GateUnit next;
            if (ok && gate_unit(a, u.unit + gridDim.x, &next)) begin(next);
        }
        const int rb = warp % 4, t = rb * 32 + lane;
        const int cb = warp / 4;
        if (cb <= rb) {
            const Sum2 mine = gt.sum(t);
            const bool live = t < u.left;
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
            rows[cb][t] = sum;
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
            columns[rb][cb * 32 + lane] = z[0];   // (lane's bits chose column `lane`)
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp < 4) {   // a warp takes 32 steps; the others go on to the next chunk
            const int t = warp * 32 + lane;
            float d = 0.f, below = 0.f, here = 0.f;
            for (int r = warp; r < 4; ++r) d += columns[r][t];
            // Rows' sums over the blocks before this one: of the rows below, whole; of its own, from step u on.
            for (int cb = 0; cb < warp; ++cb) {
                here += rows[cb][t];
                for (int r = warp + 1; r < 4; ++r) below += rows[cb][r * 32 + lane];
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
            if (t < u.left) store_any(a.dg, a.gate16, (size_t)u.row0 + (size_t)t * a.Hv, d + below + from + before + whole);
        }
        more = gate_unit(a, u.unit + gridDim.x, &u);
    }
    if (warp == 12) {
        if (elect_one() && (!ok || *gone)) {
            for (uint64_t *x : {&sh.q, &sh.k, &sh.v}) drain_wait(x, (loaded - 1) & 1, a.ctl);
            if (sent) drain_wait(&sh.o, (sent - 1) & 1, a.ctl);
            drain_products(&sh.drain, a.ctl);
        }
        __syncwarp();
    }
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tm) : "memory");
}

}  // namespace qs
