// delta_fwd_tc.cuh -- forward of the gated delta rule on the tensor cores.
//
// One CTA walks the chunks of one (sequence, value head).  Everything that the
// chain of states goes through is laid out transposed: the state M^T [dv][dk], the
// errors e^T [dv][t] and so on have one value row dv per tensor-memory lane:
// threads own rows of every product of the chain, and no value crosses threads
// between two of them.  Four warpgroups:
//
//   walk    two warpgroups: [X Y] = M^T [K;Q]^T;  e = (v - exp(G) X) T^T;
//           dM = (beta left e)^T K;  o = scale exp(G) Y + U P^T.  Each converts half of
//           the columns between two products; what the chain does not wait for (o, the
//           stores) runs while the products do
//   prep    two warpgroups, one chunk ahead (delta_prep.cuh)
//
// The state stays in the registers of `walk` (fp32, half of dk each): adding
// dM to it there rounds once, where adding up in the tensor cores would cut off the
// state's last bit with every one of the product's passes.
//
// Bound: the chain's latency.  Per chunk of 64 steps it is three products after each
// other (D = 128: 4.2 + 1 + 2.1 MFLOP, in 3 to 6 passes), with conversions to terms
// between them.  A product of 64 columns takes the tensor cores as long as one of
// 128, which is why X and Y are one.  Conversions run in pieces of 16 columns: code
// that stays in the instruction cache while four roles run, and few registers.
// Measured (bfloat16): 8 x 4096 x 16 x 128, 128 walks of 64 chunks, 375 us, 5.9 us a
// chunk (487 us with the states and errors saved: 1.2 GB, 2.5 TB/s); 1 x 131072 x 16 x 64
// in 19 segments, with their sums and join, 2.11 ms; 8 x 4096 x 16 x 128 fp32 904 us.  Under the
// profiler the tensor pipe is busy for 22% of the time, issue slots for 35% of the GPU's (43% of an SM with a walk), and
// stalls are loads from tensor memory, the walk's barriers and the waits for products.
#pragma once

#include "delta_prep.cuh"

namespace qs {

// Tensor-memory columns of the forward walk.
namespace fwd_tmem {
constexpr uint32_t D = 0;      // [X Y] (64 + 64), later dM (128)
constexpr uint32_t SP = 128;   // terms of M (3 x 64); then of v - exp(G) X (3 x 32, with fp32 inputs later of U) and of beta left e (3 x 32)
constexpr uint32_t X = 320;    // e, then (bfloat16 inputs) U: each 32 columns of e give way to their own terms
constexpr uint32_t O = 384;    // scale exp(G) Y, then o
constexpr uint32_t G = 448;    // Gram products
}  // namespace fwd_tmem

struct UAt {   // U's columns: K step k of a term
    bool early;
    __device__ __forceinline__ uint32_t operator()(int k) const { return early ? (uint32_t)(k / 2 * 32 + k % 2 * 8) : (uint32_t)(k * 8); }
};

// SUM: sums a segment up (delta_prep.cuh) and writes no o.
template <typename T, int NT, int DK, bool SUM>
__global__ void __launch_bounds__(kWalkThreads, 1)
    delta_fwd_tc_kernel(const __grid_constant__ DeltaArgs a, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap vmap) {
    constexpr int PT = NT == 1 ? 2 : 3;   // terms of what only o is made of: two leave out 2^-15 at most, bfloat16's own rounding is 2^-9
    using L = WalkLayout<NT, DK, PT>;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024u - smem_addr(raw) % 1024u) % 1024u);
    const uint32_t sm32 = smem_addr(sm);
    WalkBars &bar = *reinterpret_cast<WalkBars *>(sm + L::BARS_AT);
    volatile int *gone = &bar.gone;
    const ChunkGates *gates = reinterpret_cast<const ChunkGates *>(sm + L::GATES_AT);

    const Walk walk = walk_of<SUM, false>(a);
    const int head = walk.head;
    const long long n = walk.n;
    Seq seq = seq_of(a, n);
    if (a.segs > 1) seq = segment_of(a, seq, walk.seg);
    const int chunks = (int)((seq.len + DC - 1) / DC);
    const int wg = warp_uniform(threadIdx.x / 128), tid = threadIdx.x % 128, warp = warp_uniform(threadIdx.x / 32);
    const uint32_t tm = walk_setup<L>(bar, sm32);

    if (wg >= 2) {
        walk_prep<T, NT, DK, PT, false>(a, a.v, a.sv, bar, sm, seq, chunks, head, tm, fwd_tmem::G);
    } else {
        constexpr int HALF = DK / 2;             // columns of the state per thread
        constexpr bool kEarly = NT == 1;         // U has a place of its own: the next chunk need not wait for o
        const uint32_t tl = tm + ((uint32_t)(warp % 4 * 32) << 16);   // this warp's lanes
        const int dv = tid, col0 = wg * HALF;
        const WalkRow row(a, walk, tid);
        const bool in = row.in;
        const size_t state = ((size_t)n * a.Hv + head) * a.Dk * a.Dv + dv, step = (size_t)a.Hv * a.Dv;
        const long long row0 = seq.b * a.S + seq.s0;
        if (NT == 1 && warp == 0 && elect_one())
            for (int i = 0; i < L::KS; ++i) fetch_rows<L, false>(a, &kmap, &qmap, &vmap, bar, sm, seq, i, chunks, head);
        __syncwarp();
        float2 m[HALF / 2];
        float whole = 0.f;
        bool ok = true;   // none of this thread's waits has run out
        const float *from = a.segs > 1 ? a.seg_m + walk.at * a.Dk * a.Dv + dv : a.init ? a.init + state : nullptr;
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
            float v;
            if (SUM) v = row.map && col0 + i == row.row ? 1.f : 0.f;
            else v = from && in && col0 + i < a.Dk ? __ldg(from + (size_t)(col0 + i) * a.Dv) : 0.f;
            if (i % 2) m[i / 2].y = v;
            else m[i / 2].x = v;
        }

        // The state after a chunk whose dM is in tensor memory.
        auto add_dm = [&](int p) {   // columns 16p ..
            uint32_t r[16];
            tmem_ld16(tl + fwd_tmem::D + col0 + p * 16, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i)
                m[p * 8 + i] = fma2(make_float2(whole, whole), m[p * 8 + i], make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])));
        };
        // o of chunk c, this warpgroup's half of the steps.
        auto write_o = [&](int c) {
            ok &= tc_wait_warp(&bar.o, c & 1, gone, a.ctl);
            const int left = (int)min((long long)DC, seq.len - (long long)c * DC);
            T *out = static_cast<T *>(a.o) + ((size_t)(row0 + (long long)c * DC + wg * 32) * a.Hv + head) * a.Dv + dv;
#pragma unroll 1
            for (int h = wg * 32; h < wg * 32 + 32; h += 16, out += 16 * step) {
                uint32_t r[16];
                tmem_ld16(tl + fwd_tmem::O + h, r);
                tmem_wait_ld();
                store_columns(out, step, left - h, in, reinterpret_cast<const float *>(r));
            }
        };

#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const uint32_t rows = sm32 + c % L::KS * L::ROWS, tile_t = sm32 + L::T_AT + c % L::S * L::SLOT, tile_p = tile_t + L::P_IN;
            const ChunkGates &gt = gates[c & 3];
            const int left = (int)min((long long)DC, seq.len - (long long)c * DC);
            if (c > 0) {
                ok &= tc_wait_warp(&bar.s, (c - 1) & 1, gone, a.ctl);
                if (NT == 1 && warp == 0 && elect_one() && ok)   // the last chunk's rows are done with (prep waits for these before it fills T)
                    fetch_rows<L, false>(a, &kmap, &qmap, &vmap, bar, sm, seq, c - 1 + L::KS, chunks, head);
                __syncwarp();
            }
            if (!SUM && !kEarly && c > 0) ok &= tc_wait_warp(&bar.o, (c - 1) & 1, gone, a.ctl);
#pragma unroll
            for (int p = 0; p < HALF / 16; ++p) {
                if (c > 0) add_dm(p);
                put_terms3(tl + fwd_tmem::SP + (col0 + p * 16) / 2, 64, m + p * 8);
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, 256);
            ok &= tc_wait_warp(&bar.full[c % L::S], (c / L::S) & 1, gone, a.ctl);
            if (NT == 1) ok &= tc_wait_warp(&bar.rows[c % L::KS], (c / L::KS) & 1, gone, a.ctl);   // (V is read by all)
            whole = gt.whole;
            if (warp == 0 && elect_one() && ok) {
                tc_fence_after();
                issue_ts<3, NT, 2, DK / 16>(tm + fwd_tmem::D, tm + fwd_tmem::SP, 64, smem_desc(rows, 16, 1024), L::KQ_TERM,
                                            mma_desc(128, SUM ? 64 : 128), TmemK(), KMajor());
                mma_commit(&bar.x);
            }
            __syncwarp();
            // While the products run: the state that entered the chunk (half of it now, half behind
            // the next product), and the last chunk's o.
            auto write_carry = [&](int part) {
                if (SUM || !a.carries) return;
                float *out = a.carries + ((size_t)(seq.slot0 + c) * a.Hv + head) * a.Dk * a.Dv + (size_t)col0 * a.Dv + dv;
                if (in)
#pragma unroll
                    for (int i = 0; i < HALF; ++i, out += a.Dv)
                        if (i / (HALF / 2) == part && col0 + i < a.Dk) *out = i % 2 ? m[i / 2].y : m[i / 2].x;
                __syncwarp();
            };
            write_carry(0);
            if (!SUM && c > 0) write_o(c - 1);
            ok &= tc_wait_warp(&bar.x, c & 1, gone, a.ctl);
#pragma unroll 1
            for (int h = wg * 32; h < wg * 32 + 32; h += 16) {   // v - exp(G) X
                uint32_t r[16];
                float v[16];
                float2 e[8];
                tmem_ld16(tl + fwd_tmem::D + h, r);
                third_column<NT>(sm + c % L::KS * L::ROWS + L::V_AT, dv, h, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    e[i] = fma2(make_float2(-__uint_as_float(r[2 * i]), -__uint_as_float(r[2 * i + 1])),
                                *reinterpret_cast<const float2 *>(&gt.grown[h + 2 * i]),
                                SUM && row.map ? make_float2(0.f, 0.f) : make_float2(v[2 * i], v[2 * i + 1]));
                put_terms3(tl + fwd_tmem::SP + h / 2, 32, e);
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, 256);
            if (warp == 0 && elect_one() && ok) {
                tc_fence_after();
                issue_ts<3, 3, 2, DC / 16>(tm + fwd_tmem::X, tm + fwd_tmem::SP, 32, smem_desc(tile_t, 16, 1024), TILE,
                                           mma_desc(128, 64), TmemK(), KMajor1());
                mma_commit(&bar.e);
            }
            __syncwarp();
            if (!SUM) {   // Y moves, so that dM can take its place and o add up on it
#pragma unroll 1
                for (int h = wg * 32; h < wg * 32 + 32; h += 16) {
                    uint32_t r[16];
                    tmem_ld16(tl + fwd_tmem::D + 64 + h, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 g = mul2(*reinterpret_cast<const float2 *>(&gt.grown[h + 2 * i]), make_float2(a.scale, a.scale));
                        const float2 y = mul2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), g);
                        r[2 * i] = __float_as_uint(y.x), r[2 * i + 1] = __float_as_uint(y.y);
                    }
                    tmem_st16(tl + fwd_tmem::O + h, r);
                }
            }
            write_carry(1);
            ok &= tc_wait_warp(&bar.e, c & 1, gone, a.ctl);
            const int h0 = wg * 32;
            float2 u[16];   // beta e
            {
                uint32_t r[32];   // (U takes the place of 32 columns of e: all are read first)
                tmem_ld32(tl + fwd_tmem::X + h0, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
            }
            if (!SUM && a.errors && in) {
                float *eo = a.errors + ((size_t)(row0 + (long long)c * DC + h0) * a.Hv + head) * a.Dv + dv;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (h0 + i < left) eo[i * step] = i % 2 ? u[i / 2].y : u[i / 2].x;
            }
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 2; ++q) {   // the state's update first: the chain waits for it
                float2 k[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int s = q * 16 + 2 * i;
                    u[s / 2] = mul2(u[s / 2], *reinterpret_cast<const float2 *>(&gt.beta[h0 + s]));
                    k[i] = mul2(u[s / 2], *reinterpret_cast<const float2 *>(&gt.left[h0 + s]));
                }
                put_terms3(tl + fwd_tmem::SP + 96 + (h0 + q * 16) / 2, 32, k);
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, 256);
            if (warp == 0 && elect_one() && ok) {
                tc_fence_after();
                issue_ts<3, NT, 2, DC / 16>(tm + fwd_tmem::D, tm + fwd_tmem::SP + 96, 32, smem_desc(rows, 2 * TILE, 1024), L::KQ_TERM,
                                            mma_desc(128, DK, false, true), TmemK(), MNMajor());
                mma_commit(&bar.s);
                if (SUM) mma_commit(&bar.empty[c % L::S]);
            }
            __syncwarp();
            if (!SUM) {   // U, for o
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t t[PT][8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t p[3];
                        split2<PT>(u[q * 8 + i], p);
#pragma unroll
                        for (int j = 0; j < PT; ++j) t[j][i] = p[j];
                    }
#pragma unroll
                    for (int j = 0; j < PT; ++j)
                        tmem_st8(tl + (kEarly ? fwd_tmem::X + h0 + j * 16 : fwd_tmem::SP + j * 32 + h0 / 2) + q * 8, t[j]);
                }
                tmem_wait_st();
                tc_fence_before();
                named_bar_sync(1, 256);
                if (warp == 0 && elect_one() && ok) {
                    tc_fence_after();
                    issue_ts<PT, PT, PT - 1, DC / 16>(tm + fwd_tmem::O, tm + (kEarly ? fwd_tmem::X : fwd_tmem::SP), kEarly ? 16 : 32,
                                                      smem_desc(tile_p, 16, 1024), TILE, mma_desc(128, 64), UAt{kEarly},
                                                      KMajor1(), true);
                    mma_commit(&bar.o);
                    mma_commit(&bar.empty[c % L::S]);
                }
                __syncwarp();
            }
        }
        if (chunks > 0) {
            ok &= tc_wait_warp(&bar.s, (chunks - 1) & 1, gone, a.ctl);
#pragma unroll
            for (int p = 0; p < HALF / 16; ++p) add_dm(p);
            if (!SUM) write_o(chunks - 1);
        }
        if (SUM) {
            if (in)
#pragma unroll
                for (int i = 0; i < HALF; ++i)
                    if (col0 + i < a.Dk) *row.sum_out(a, walk, col0 + i) = i % 2 ? m[i / 2].y : m[i / 2].x;
        } else if (a.fin && in && walk.seg == a.segs - 1)
#pragma unroll
            for (int i = 0; i < HALF; ++i)
                if (col0 + i < a.Dk) a.fin[state + (size_t)(col0 + i) * a.Dv] = i % 2 ? m[i / 2].y : m[i / 2].x;
        if (warp == 0 && elect_one() && (!ok || *gone)) drain_walk<L>(bar, a.ctl);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free_all(tm);
}

}  // namespace qs
