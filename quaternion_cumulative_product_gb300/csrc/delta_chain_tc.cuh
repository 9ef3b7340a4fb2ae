// delta_chain_tc.cuh -- backward of the gated delta rule on the tensor cores: the
// chain of the states' cotangents, from the last chunk to the first.
//
// One CTA walks the chunks of one (sequence, value head) in reverse, laid out as the
// forward walk (delta_fwd_tc.cuh): dM^T [dv][dk] in registers, one value row per
// thread.  With T = (1 + diag(beta) A)^-1:
//
//     R = dO^T P              (only the chunk's own inputs: runs while dM' is converted)
//     X = dM'^T K^T
//     w = (exp(G_C - G) X + R) T
//     dM = exp(G_C) dM' + (scale exp(G) dO)^T Q - (exp(G) beta w)^T K
//
// Two warpgroups walk (half of the columns each between two products; w's part of the
// update one, dO's the other), two prepare, as in the forward (delta_prep.cuh).
//
// T and P are read across their rows (MN-major), dO^T as an MN-major left operand.
//
// Bound: the chain's latency, as in the forward (dM = (..) Q - (..) K is one product more).
// Measured: 8 x 4096 x 16 x 128 bfloat16 480 us, dM' of every chunk and w written (0.8 GB,
// 1.7 TB/s); tensor pipe 23%, issue slots 36%.  4 x 1000 x 8 x 64 fp32, in segments:
// 49 us, and 52 us for the segments' sums.
#pragma once

#include "delta_prep.cuh"

namespace qs {

namespace chain_tmem {
constexpr uint32_t D = 0;      // the update of dM (128)
constexpr uint32_t SP = 128;   // terms of dM' (3 x 64); then of X + R, later scale exp(G) dO (3 x 32), and of -exp(G) beta w (3 x 32)
constexpr uint32_t X = 320;    // X, then w
constexpr uint32_t R = 384;
constexpr uint32_t G = 448;
}  // namespace chain_tmem

// SUM: sums a segment up (delta_prep.cuh) and writes neither dM' nor w.
template <typename T, int NT, int DK, bool SUM>
__global__ void __launch_bounds__(kWalkThreads, 1)
    delta_chain_tc_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap omap) {
    using L = WalkLayout<NT, DK, 3>;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024u - smem_addr(raw) % 1024u) % 1024u);
    const uint32_t sm32 = smem_addr(sm);
    WalkBars &bar = *reinterpret_cast<WalkBars *>(sm + L::BARS_AT);
    volatile int *gone = &bar.gone;
    const ChunkGates *gates = reinterpret_cast<const ChunkGates *>(sm + L::GATES_AT);

    const Walk walk = walk_of<SUM, true>(a);
    const int head = walk.head;
    const long long n = walk.n;
    Seq seq = seq_of(a, n);
    if (a.segs > 1) seq = segment_of(a, seq, walk.seg);
    const int chunks = (int)((seq.len + DC - 1) / DC);
    const int wg = warp_uniform(threadIdx.x / 128), tid = threadIdx.x % 128, warp = warp_uniform(threadIdx.x / 32);
    const uint32_t tm = walk_setup<L>(bar, sm32);

    if (wg >= 2) {
        const qsh::Strides so = {(long long)a.S * a.Hv * a.Dv, (long long)a.Hv * a.Dv, a.Dv};
        walk_prep<T, NT, DK, 3, true>(a, a.d_o, so, bar, sm, seq, chunks, head, tm, chain_tmem::G);
    } else {
        constexpr int HALF = DK / 2;             // columns of dM per thread
        const uint32_t tl = tm + ((uint32_t)(warp % 4 * 32) << 16);   // this warp's lanes
        const int dv = tid, col0 = wg * HALF;
        const WalkRow row(a, walk, tid);
        const bool in = row.in;
        const size_t state = ((size_t)n * a.Hv + head) * a.Dk * a.Dv + dv, step = (size_t)a.Hv * a.Dv;
        const long long row0 = seq.b * a.S + seq.s0;
        if (NT == 1 && warp == 0 && elect_one())
            for (int i = 0; i < L::KS; ++i) fetch_rows<L, true>(a, &kmap, &qmap, &omap, bar, sm, seq, i, chunks, head);
        __syncwarp();
        float2 m[HALF / 2];
        float whole = 0.f;
        bool ok = true;   // none of this thread's waits has run out
        const float *from = a.segs > 1 ? a.seg_m + walk.at * a.Dk * a.Dv + dv : a.d_final ? a.d_final + state : nullptr;
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
            float v;
            if (SUM) v = row.map && col0 + i == row.row ? 1.f : 0.f;
            else v = from && in && col0 + i < a.Dk ? __ldg(from + (size_t)(col0 + i) * a.Dv) : 0.f;
            if (i % 2) m[i / 2].y = v;
            else m[i / 2].x = v;
        }
        auto add_update = [&](int p) {   // columns 16p ..
            uint32_t r[16];
            tmem_ld16(tl + chain_tmem::D + col0 + p * 16, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m[p * 8 + i] = fma2(make_float2(whole, whole), m[p * 8 + i], make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
        };

#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            const int c = chunks - 1 - it;
            const uint32_t rows = sm32 + it % L::KS * L::ROWS, tile_t = sm32 + L::T_AT + it % L::S * L::SLOT, tile_p = tile_t + L::P_IN;
            const ChunkGates &gt = gates[it & 3];
            const int left = (int)min((long long)DC, seq.len - (long long)c * DC);
            if (it > 0) {
                ok &= tc_wait_warp(&bar.s, (it - 1) & 1, gone, a.ctl);
                if (NT == 1 && warp == 0 && elect_one() && ok)   // the last chunk's rows are done with (prep waits for these before it fills T)
                    fetch_rows<L, true>(a, &kmap, &qmap, &omap, bar, sm, seq, it - 1 + L::KS, chunks, head);
                __syncwarp();
            }
            ok &= tc_wait_warp(&bar.full[it % L::S], (it / L::S) & 1, gone, a.ctl);
            if (NT == 1) ok &= tc_wait_warp(&bar.rows[it % L::KS], (it / L::KS) & 1, gone, a.ctl);   // (dO is read by all)
            if (warp == 0 && elect_one() && ok) {   // R = dO^T P
                issue_ss<NT, 3, 2, DC / 16>(tm + chain_tmem::R, smem_desc(rows + L::V_AT, TILE, 1024), L::V_TERM,
                                            smem_desc(tile_p, 16, 1024), TILE, mma_desc(128, 64, true, true), MNMajor(), MNMajor());
            }
            __syncwarp();
#pragma unroll
            for (int p = 0; p < HALF / 16; ++p) {
                if (it > 0) add_update(p);
                put_terms3(tl + chain_tmem::SP + (col0 + p * 16) / 2, 64, m + p * 8);
            }
            whole = gt.whole;
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, 256);
            if (warp == 0 && elect_one() && ok) {
                tc_fence_after();
                issue_ts<3, NT, 2, DK / 16>(tm + chain_tmem::X, tm + chain_tmem::SP, 64, smem_desc(rows, 16, 1024), L::KQ_TERM,
                                            mma_desc(128, 64), TmemK(), KMajor());
                mma_commit(&bar.x);
            }
            __syncwarp();
            auto write_ds = [&](int part) {   // dM', half of it behind each of two products
                if (SUM) return;
                float *out = a.ds + ((size_t)(seq.slot0 + c) * a.Hv + head) * a.Dk * a.Dv + (size_t)col0 * a.Dv + dv;
                if (in)
#pragma unroll
                    for (int i = 0; i < HALF; ++i, out += a.Dv)
                        if (i / (HALF / 2) == part && col0 + i < a.Dk) *out = i % 2 ? m[i / 2].y : m[i / 2].x;
                __syncwarp();
            };
            write_ds(0);
            ok &= tc_wait_warp(&bar.x, it & 1, gone, a.ctl);
#pragma unroll 1
            for (int h = wg * 32; h < wg * 32 + 32; h += 16) {
                uint32_t r[16], y[16];
                float2 e[8];
                tmem_ld16(tl + chain_tmem::X + h, r);
                tmem_ld16(tl + chain_tmem::R + h, y);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    e[i] = fma2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                                *reinterpret_cast<const float2 *>(&gt.left[h + 2 * i]),
                                SUM && row.map ? make_float2(0.f, 0.f) : make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1])));
                put_terms3(tl + chain_tmem::SP + h / 2, 32, e);
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, 256);
            if (warp == 0 && elect_one() && ok) {
                tc_fence_after();
                issue_ts<3, 3, 2, DC / 16>(tm + chain_tmem::X, tm + chain_tmem::SP, 32, smem_desc(tile_t, 16, 1024), TILE,
                                           mma_desc(128, 64, false, true), TmemK(), MNMajor());
                mma_commit(&bar.e);
                mma_commit(&bar.empty[it % L::S]);
            }
            __syncwarp();
            write_ds(1);
            ok &= tc_wait_warp(&bar.e, it & 1, gone, a.ctl);
            if (wg == 0) {
#pragma unroll 1
                for (int h = 0; h < DC; h += 16) {   // -exp(G) beta w
                    uint32_t r[16];
                    float2 z[8];
                    tmem_ld16(tl + chain_tmem::X + h, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        z[i] = mul2(mul2(make_float2(-__uint_as_float(r[2 * i]), -__uint_as_float(r[2 * i + 1])),
                                         *reinterpret_cast<const float2 *>(&gt.beta[h + 2 * i])),
                                    *reinterpret_cast<const float2 *>(&gt.grown[h + 2 * i]));
                    put_terms3(tl + chain_tmem::SP + 96 + h / 2, 32, z);
                }
            } else {   // scale exp(G) dO, where the terms of X + R were
#pragma unroll 1
                for (int h = 0; h < DC; h += 16) {
                    float v[16];
                    float2 z[8];
                    third_column<NT>(sm + it % L::KS * L::ROWS + L::V_AT, dv, h, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        z[i] = mul2(mul2(SUM && row.map ? make_float2(0.f, 0.f) : make_float2(v[2 * i], v[2 * i + 1]), *reinterpret_cast<const float2 *>(&gt.grown[h + 2 * i])),
                                    make_float2(a.scale, a.scale));
                    put_terms3(tl + chain_tmem::SP + h / 2, 32, z);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, 256);
            if (warp == 0 && elect_one() && ok) {
                tc_fence_after();
                const uint32_t id = mma_desc(128, DK, false, true);
                // Both products' small terms, then both products' first ones: a pass cuts off the last
                // bit of what the accumulator holds by then.
#pragma unroll 1
                for (int n = 0; n < 4; ++n)
                    issue_ts<3, NT, 2, DC / 16>(tm + chain_tmem::D, tm + chain_tmem::SP + n % 2 * 96, 32,
                                                smem_desc(n % 2 ? rows : rows + TILE, 2 * TILE, 1024), L::KQ_TERM, id, TmemK(), MNMajor(),
                                                n > 0, n < 2 ? kSmallPairs : kFirstPair);
                mma_commit(&bar.s);
            }
            __syncwarp();
            if (!SUM) {   // w and dv, half of the steps each, while the products run
                const int h0 = wg * 32;
                const size_t at = ((size_t)(row0 + (long long)c * DC + h0) * a.Hv + head) * a.Dv + dv;
                float *wo = a.w + at;
                T *vo = static_cast<T *>(a.dv) + at;
#pragma unroll 1
                for (int h = h0; h < h0 + 32; h += 16, wo += 16 * step, vo += 16 * step) {
                    uint32_t r[16];
                    tmem_ld16(tl + chain_tmem::X + h, r);
                    tmem_wait_ld();
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(r[i]);
                    store_columns(wo, step, left - h, in, x);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] *= gt.beta[h + i];
                    store_columns(vo, step, left - h, in, x);
                }
                tc_fence_before();
            }
        }
        if (chunks > 0) {
            ok &= tc_wait_warp(&bar.s, (chunks - 1) & 1, gone, a.ctl);
#pragma unroll
            for (int p = 0; p < HALF / 16; ++p) add_update(p);
        }
        if (SUM) {
            if (in)
#pragma unroll
                for (int i = 0; i < HALF; ++i)
                    if (col0 + i < a.Dk) *row.sum_out(a, walk, col0 + i) = i % 2 ? m[i / 2].y : m[i / 2].x;
        } else if (a.d_init && in && walk.seg == 0)
#pragma unroll
            for (int i = 0; i < HALF; ++i)
                if (col0 + i < a.Dk) a.d_init[state + (size_t)(col0 + i) * a.Dv] = i % 2 ? m[i / 2].y : m[i / 2].x;
        if (warp == 0 && elect_one() && (!ok || *gone)) drain_walk<L>(bar, a.ctl);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free_all(tm);
}

}  // namespace qs
