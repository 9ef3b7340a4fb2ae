// delta_bwd_tc.cuh -- backward of the gated delta rule on the tensor cores: the
// gradients of one chunk from the state that enters it, the cotangent of the
// state that leaves it, its errors e and its w.
//
// One CTA per (chunk, value head), four warpgroups that share the 128 rows of each
// product (each takes a quarter of the columns).  Rows of queries and of keys are
// stacked, so that one product serves both:
//
//     R = [dO; dV] M^T            the states' part of dq and of row
//     S = [dO; dV] U^T            X, Y (64 + 64 rows) once the decays are on
//     C = U dM'^T                 the states' part of col (rows 64 .. 127)
//     I = [X; Y] K                the chunk's part of dq and of row
//     J = [X; Y]^T [Q; K]         the chunk's part of col
//     H = [Q; K] K^T              for dg
//
// (names as in delta_common.cuh).  I and J have accumulators of their own, and are added
// to R and C, with the decays of their rows, in registers: adding up on R and C in the
// tensor cores would cut off their last bit with each of 24 to 48 passes.  The stacked left operand is in tensor memory, the
// others in shared memory; [X;Y] is a K-major operand in one product and an MN-major
// one in the other.  C's left operands have 64 rows; they stand in rows 64 .. 127 of
// 128 (what lies before them in shared memory fills the others, which nobody
// reads), so that a key's row and its col meet in one thread.
//
// Terms: CT bfloat16 terms per computed value: three (fp32 precision) where any
// output is fp32; two (2^-15 of a product left out at most, rms 2^-17.8) where outputs and
// gates are bfloat16, whose own rounding is 2^-9.  dg bears it too: no two of its sums cancel.
//
// Bound: the latency of its phases (loads, conversions, five products), one CTA per
// SM.  Global loads run along the rows (a warp covers whole lines): loads by the
// thread that owns a row touch 32 lines each, and were half of the kernel's time.
// Measured at 8 x 4096 x 16 x 128 bfloat16 (8192 CTAs): 777 us with two terms (bfloat16 gates), 904 us
// with three (fp32 gates); of a CTA's 29k clocks about 13k go to the loads and 16k to conversions,
// products and stores.  2.2 GB, 2.9 TB/s; tensor pipe 20%, issue slots 32%.  H and Z are 43 and 36 us
// of that; without them dg cancels (delta_common.cuh).  Without H and Z, M and dM' copied in bulk over
// the place of their terms, instead of loaded by all threads: 727 against 732 us, but 934 against 868 with three terms.
#pragma once

#include "delta_prep.cuh"

namespace qs {

constexpr int kChunkThreads = 512;

// Sums in shared memory (floats).
namespace row_sums {
constexpr int A = 0;                // [warpgroup][128] a's parts of a query's and a key's row (before that [64] dbeta)
constexpr int B = A + 4 * 128;      // [warpgroup][64] b's parts
constexpr int TOTAL = B + 4 * 64;   // [8][64] Z's columns over eight steps each
constexpr int Z = TOTAL + 8 * 64;   // [2][64] Z's part of dg, by halves of its columns
constexpr int MD = Z + 2 * 64;      // [16] exp(G_C) <M, dM'> by warps
constexpr int COUNT = MD + 16;
}  // namespace row_sums

template <int NT, int CT, int DK>
struct ChunkLayout {
    static constexpr int HALVES = DK / 64;
    static constexpr int SH = NT == 1 ? 2 : 1;                           // halves of dv held at a time
    static constexpr bool BOTH = NT == 1 && CT == 2;                     // M and dM' have room side by side
    static constexpr uint32_t QK_TERM = HALVES * 2 * TILE;
    static constexpr uint32_t M_HALF = DK * 128, M_TERM = SH * M_HALF;   // M, dM': [term][half of dv][DK rows]
    static constexpr uint32_t A_HALF = 2 * TILE, A_TERM = SH * A_HALF;   // [dO; dV] on its way: [term][half of dv][128 rows]
    static constexpr uint32_t QK_AT = 0, U_AT = NT * QK_TERM;            // U: [term][half of dv][64 rows]
    static constexpr uint32_t M_AT = U_AT + CT * 2 * TILE;
    static constexpr uint32_t max2(uint32_t a, uint32_t b) { return a > b ? a : b; }
    static constexpr uint32_t M_BYTES = max2(CT * M_TERM, max2(CT * 2 * TILE, BOTH ? 0 : CT * A_TERM));   // later [X;Y]: [term][128 rows]
    static constexpr uint32_t DM_AT = BOTH ? M_AT + M_BYTES : M_AT;
    static constexpr uint32_t A_AT = DM_AT;
    static constexpr uint32_t GATES_AT = BOTH ? DM_AT + max2(CT * M_TERM, CT * A_TERM) : M_AT + M_BYTES;
    static constexpr uint32_t ROWS_AT = GATES_AT + sizeof(ChunkGates);
    static constexpr uint32_t BARS_AT = ROWS_AT + row_sums::COUNT * 4;
    static constexpr uint32_t NEED = BARS_AT + 256 + 1024;
    static constexpr uint32_t BYTES = NEED > 117760 ? NEED : 117760;     // one CTA per SM: it takes all of the tensor memory
    static_assert(BYTES <= 232448, "227 KB of shared memory");
};

namespace bwd_tmem {
constexpr uint32_t A = 0;      // terms (3 x 64) of [dO; dV]
constexpr uint32_t S = 192;    // [dO; dV] U^T (64)
constexpr uint32_t R = 256, C = 384;
constexpr uint32_t I = 0, J = 128;   // over A and S
}  // namespace bwd_tmem

// H's columns: beside two terms of A, or over A once that is done with.
template <int CT>
constexpr uint32_t kGramAt = CT == 2 ? 128 : 0;

struct ChunkBars {
    uint64_t m, s, e, r, drain;
    uint32_t tmem;
    int gone;
};

// Eight fp32 values at a row's unit u as CT terms, `term` bytes apart.
template <int CT>
__device__ __forceinline__ void unit_terms(uint32_t at, uint32_t term, const float4 p, const float4 q) {
    uint32_t s[4][3];
    split2<CT>(p.x, p.y, s[0]), split2<CT>(p.z, p.w, s[1]), split2<CT>(q.x, q.y, s[2]), split2<CT>(q.z, q.w, s[3]);
#pragma unroll
    for (int j = 0; j < CT; ++j) {
        const uint32_t v[4] = {s[0][j], s[1][j], s[2][j], s[3][j]};
        st_shared16(at + j * term, v);
    }
}

__device__ __forceinline__ float4 scaled(const float4 v, float f) { return make_float4(v.x * f, v.y * f, v.z * f, v.w * f); }

template <typename T, int NT, int CT, int DK>
__global__ void __launch_bounds__(kChunkThreads, 1) delta_chunk_tc_kernel(const __grid_constant__ DeltaArgs a) {
    using L = ChunkLayout<NT, CT, DK>;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024u - smem_addr(raw) % 1024u) % 1024u);
    const uint32_t sm32 = smem_addr(sm);
    ChunkBars &bar = *reinterpret_cast<ChunkBars *>(sm + L::BARS_AT);
    ChunkGates &gt = *reinterpret_cast<ChunkGates *>(sm + L::GATES_AT);
    float *rows = reinterpret_cast<float *>(sm + L::ROWS_AT);   // row_sums
    volatile int *gone = &bar.gone;
    bool ok = true;   // none of this thread's waits has run out

    const int head = blockIdx.x % a.Hv, kh = head / (a.Hv / a.Hk);
    Seq seq;
    long long c;
    if (!chunk_of(a, blockIdx.x / a.Hv, &seq, &c)) return;
    const long long t0 = c * DC, row0 = seq.b * a.S + seq.s0 + t0;
    const int left = (int)min((long long)DC, seq.len - t0);
    const int wg = warp_uniform(threadIdx.x / 128), warp = warp_uniform(threadIdx.x / 32);
    const int tid = threadIdx.x % 128, lane = threadIdx.x % 32, t = tid % 64;
    const bool live = t < left, keys = warp % 4 >= 2;   // this thread's row of the products: a query's or a key's
    const size_t at0 = ((size_t)(seq.slot0 + c) * a.Hv + head) * a.Dk * a.Dv;
    const int dvh = a.Dv <= 64 ? 1 : 2;                 // halves of dv in use

    if (threadIdx.x == 0) {
        for (uint64_t *b : {&bar.m, &bar.s, &bar.e, &bar.r, &bar.drain}) mbar_init(b, 1);
        *gone = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc_all(&bar.tmem);
    if (warp == 1) warp_gates(gt, read_gates(a, seq, t0, head));
    {   // Q by half of the threads, K by the others
        const int w = wg / 2;
        load_rows<T, NT, DK, 256>(sm32 + L::QK_AT + w * TILE, 2 * TILE, L::QK_TERM, w ? a.k : a.q, w ? a.sk : a.sq, seq, t0, kh, a.Dk,
                                  threadIdx.x % 256);
    }

    // M and dM' as they are read: JT units of eight values per thread, unit j of a thread at
    // the same place of either.
    constexpr int UNITS = 8 * L::SH, JT = DK * 16 / kChunkThreads, JR = JT * L::SH / 2;   // units per row and round; per thread and round
    auto unit_row = [&](int j) { return (int)(threadIdx.x + kChunkThreads * (j % JR)) / UNITS; };
    auto unit_x = [&](int j) { return (int)(threadIdx.x % UNITS) * 8 + j / JR * 64; };   // first value
    auto read_state = [&](const float *p, float4 (*v)[2]) {
#pragma unroll
        for (int j = 0; j < JT; ++j) {
            const int r = unit_row(j), x = unit_x(j);
            const bool in = r < a.Dk && x < a.Dv;
            const float4 *src = reinterpret_cast<const float4 *>(p + at0 + (in ? (size_t)r * a.Dv + x : 0));
            const float4 lo = __ldg(src), hi = __ldg(src + 1);
            v[j][0] = in ? lo : q_zero(), v[j][1] = in ? hi : q_zero();
        }
    };
    auto put_state = [&](uint32_t at, const float4 (*v)[2], int round) {   // the units of one round
#pragma unroll
        for (int j = 0; j < JT; ++j)
            if (j / JR == round) {
                const int r = unit_row(j), x = unit_x(j) - round * 64;
                unit_terms<CT>(at + x / 64 * L::M_HALF + swizzled(r, x % 64 / 8), L::M_TERM, v[j][0], v[j][1]);
            }
    };
    float4 m[JT][2], dm[JT][2];
    read_state(a.carries_in, m);
    if (L::BOTH) read_state(a.ds, dm);
    __syncthreads();   // the gates

    // D (+)= [dO; dV] x B, K steps k0 .. of the operand in tensor memory, B K-major.
    uint32_t tm = 0;
    auto issue_a = [&](uint32_t d, uint32_t b, uint32_t b_term, uint32_t b_half, uint32_t idesc, int k0, int halves, bool add) {
        const uint64_t base = smem_desc(b, 16, 1024);
#pragma unroll 1
        for (int i = CT - 1; i >= 0; --i)
#pragma unroll 1
            for (int j = CT - 1 - i; j >= 0; --j)
#pragma unroll 1
                for (int h = 0; h < halves; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        mma_ts(d, tm + bwd_tmem::A + i * 64 + (k0 + h * 4 + k) * 8, base + ((j * b_term + h * b_half + k * 32) >> 4), idesc, add);
                        add = true;
                    }
    };
    const uint32_t id_dk = mma_desc(128, DK), id_s = mma_desc(128, 64);
    auto issue_h = [&] {
        issue_ss<NT, NT, 2, DK / 16>(tm + kGramAt<CT>, smem_desc(sm32 + L::QK_AT, 16, 1024), L::QK_TERM,
                                     smem_desc(sm32 + L::QK_AT + TILE, 16, 1024), L::QK_TERM, id_s, KMajor(), KMajor());
    };

    // Rows: U, [dO; dV] and dbeta = <e, w>, in rounds of SH halves of dv; M alongside.
    const int rounds = (dvh + L::SH - 1) / L::SH;
#pragma unroll 1
    for (int round = 0; round < rounds; ++round) {
        constexpr int RJ = DC * UNITS / kChunkThreads;
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
            const int i = threadIdx.x + kChunkThreads * j, r = i / UNITS, x = i % UNITS * 8 + round * 64, xr = x - round * 64;
            const bool in = r < left && x < a.Dv;
            const size_t at = in ? ((size_t)(row0 + r) * a.Hv + head) * a.Dv + x : 0;
            const float4 *ep = reinterpret_cast<const float4 *>(a.errors_in + at), *wp = reinterpret_cast<const float4 *>(a.w + at);
            float4 e0 = __ldg(ep), e1 = __ldg(ep + 1), w0 = __ldg(wp), w1 = __ldg(wp + 1);
            if (!in) e0 = e1 = w0 = w1 = q_zero();
            const uint32_t stage = sm32 + L::A_AT + xr / 64 * L::A_HALF;
            if constexpr (NT == 1) {
                cp_async16_or_zero(stage + swizzled(r, xr % 64 / 8), static_cast<const T *>(a.d_o) + at, in);
            } else {
                const float4 *dp = reinterpret_cast<const float4 *>(static_cast<const float *>(a.d_o) + at);
                const float4 d0 = __ldg(dp), d1 = __ldg(dp + 1);
                unit_terms<CT>(stage + swizzled(r, xr % 64 / 8), L::A_TERM, in ? d0 : q_zero(), in ? d1 : q_zero());
            }
            float dot = dot4(e0, w0) + dot4(e1, w1);
#pragma unroll
            for (int o = UNITS / 2; o; o /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            if (threadIdx.x % UNITS == 0) rows[r] = round ? rows[r] + dot : dot;
            const float be = gt.beta[r];
            unit_terms<CT>(sm32 + L::U_AT + x / 64 * TILE + swizzled(r, x % 64 / 8), 2 * TILE, scaled(e0, be), scaled(e1, be));
            unit_terms<CT>(stage + swizzled(64 + r, xr % 64 / 8), L::A_TERM, scaled(w0, be), scaled(w1, be));
        }
        cp_async_wait_all();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (round == 0) tm = (uint32_t)warp_uniform((int)bar.tmem);
        const uint32_t tl = tm + ((uint32_t)(warp % 4 * 32) << 16);
#pragma unroll
        for (int p = 0; p < L::SH; ++p) {   // 16 values of this thread's row
            const int x = (wg * L::SH + p) * 16;
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                uint32_t v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (NT == 3 || j == 0 || keys)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint4 q = *reinterpret_cast<const uint4 *>(sm + L::A_AT + j * L::A_TERM + x / 64 * L::A_HALF + swizzled(tid, x % 64 / 8 + u));
                        v[4 * u] = q.x, v[4 * u + 1] = q.y, v[4 * u + 2] = q.z, v[4 * u + 3] = q.w;
                    }
                tmem_st8(tl + bwd_tmem::A + j * 64 + round * 32 + x / 2, v);
            }
        }
        if (L::BOTH) put_state(sm32 + L::M_AT, m, 0);   // (elsewhere than the rows on their way)
        tmem_wait_st();
        if (L::BOTH) fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
    }
    tc_fence_after();
    const uint32_t tl = tm + ((uint32_t)(warp % 4 * 32) << 16);
    if (wg == 0 && !keys && live) store_any(a.dbeta, a.gate16, (row0 + t) * a.Hv + head, rows[t]);

    // This warpgroup's quarter of an accumulator's columns: to registers, and added back.
    auto read_part = [&](uint32_t at, uint32_t *v) {
#pragma unroll
        for (int x = 0; x < DK / 4; x += 16) tmem_ld16(tl + at + wg * (DK / 4) + x, v + x);
        tmem_wait_ld();
        tc_fence_before();
    };
    auto add_part = [&](uint32_t at, const uint32_t *v) {
#pragma unroll
        for (int x = 0; x < DK / 4; x += 16) {
            uint32_t w[16];
            tmem_ld16(tl + at + wg * (DK / 4) + x, w);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) + __uint_as_float(v[x + i]));
            tmem_st8(tl + at + wg * (DK / 4) + x, w);
            tmem_st8(tl + at + wg * (DK / 4) + x + 8, w + 8);
        }
        tmem_wait_st();
    };

    // R and S; then C, dM' beside M or in its place.
    float md = 0.f;
    if (L::BOTH) {
        if (warp == 0 && elect_one() && ok) {   // (H runs while dM' is converted)
            tc_fence_after();
            issue_h();
        }
        __syncwarp();
        put_state(sm32 + L::DM_AT, dm, 0);
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0 && elect_one() && ok) {
            tc_fence_after();
            issue_a(tm + bwd_tmem::R, sm32 + L::M_AT, L::M_TERM, L::M_HALF, id_dk, 0, dvh, false);
            issue_a(tm + bwd_tmem::S, sm32 + L::U_AT, 2 * TILE, TILE, id_s, 0, dvh, false);
            mma_commit(&bar.s);
        }
    } else {
        // (A round starts its accumulators anew; the sum over the rounds is taken in registers,
        // where it rounds once: passes over a full accumulator would cut off its last bit.)
        uint32_t r0[DK / 4];
#pragma unroll 1
        for (int round = 0; round < rounds; ++round) {
            if (round) {
                ok &= tc_wait_warp(&bar.m, 0, gone, a.ctl);   // the first half of dv is done with
                read_part(bwd_tmem::R, r0);
            }
            put_state(sm32 + L::M_AT, m, round);
            fence_proxy_async_smem();
            __syncthreads();
            if (warp == 0 && elect_one() && ok) {
                tc_fence_after();
                issue_a(tm + bwd_tmem::R, sm32 + L::M_AT, L::M_TERM, L::M_HALF, id_dk, round * 4, min(dvh, L::SH), false);
                if (round + 1 < rounds) mma_commit(&bar.m);
                else {
                    issue_a(tm + bwd_tmem::S, sm32 + L::U_AT, 2 * TILE, TILE, id_s, 0, dvh, false);
                    mma_commit(&bar.s);
                }
            }
            __syncwarp();
        }
        read_state(a.ds, dm);
        ok &= tc_wait_warp(&bar.s, 0, gone, a.ctl);
        if (rounds == 2) add_part(bwd_tmem::R, r0);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < JT; ++j) md += dot4(m[j][0], dm[j][0]) + dot4(m[j][1], dm[j][1]);
    md *= gt.whole;
#pragma unroll
    for (int o = 16; o; o /= 2) md += __shfl_xor_sync(0xffffffffu, md, o);
    if (lane == 0) rows[row_sums::MD + warp] = md;
    // The CTAs of a wave run in step: all load, then all compute.  M and dM' of the CTA that
    // likely comes next on this SM go to L2 meanwhile (808 -> 734 us with two terms, 891 -> 872
    // with three; sent for before this CTA's own loads 865, with e's and w's rows 774; all without H and Z).
    if (threadIdx.x == kChunkThreads - 32 && blockIdx.x + a.sms < gridDim.x) {
        const size_t next = (size_t)(blockIdx.x + a.sms) * a.Dk * a.Dv;
        bulk_prefetch(a.ds + next, (uint32_t)(a.Dk * a.Dv) * 4);
        bulk_prefetch(a.carries_in + next, (uint32_t)(a.Dk * a.Dv) * 4);
    }
    auto issue_c = [&](int round, int halves) {   // C (+)= U dM'^T, U in rows 64 .. 127
        const uint64_t u = smem_desc(sm32 + L::U_AT - TILE, 16, 1024), d = smem_desc(sm32 + L::DM_AT, 16, 1024);
        bool add = false;
#pragma unroll 1
        for (int i = CT - 1; i >= 0; --i)
#pragma unroll 1
            for (int j = CT - 1 - i; j >= 0; --j)
#pragma unroll 1
                for (int h = 0; h < halves; ++h)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        mma_ss(tm + bwd_tmem::C, u + ((i * 2 * TILE + (round + h) * TILE + k * 32) >> 4),
                               d + ((j * L::M_TERM + h * L::M_HALF + k * 32) >> 4), id_dk, add);
                        add = true;
                    }
        if (!L::BOTH && round + 1 == rounds) issue_h();   // (A is done with: all have waited for R and S)
        mma_commit(&bar.e);
    };
    uint32_t e_phase = 0, c0[DK / 4];
    if (L::BOTH) {
        if (warp == 0 && elect_one() && ok) issue_c(0, dvh);
        __syncwarp();
        ok &= tc_wait_warp(&bar.s, 0, gone, a.ctl);
    } else {
#pragma unroll 1
        for (int round = 0; round < rounds; ++round) {
            if (round) {
                ok &= tc_wait_warp(&bar.e, 0, gone, a.ctl);
                e_phase = 1;
                read_part(bwd_tmem::C, c0);
            }
            put_state(sm32 + L::DM_AT, dm, round);
            fence_proxy_async_smem();
            __syncthreads();
            if (warp == 0 && elect_one() && ok) {
                tc_fence_after();
                issue_c(round, min(dvh, L::SH));
            }
            __syncwarp();
        }
    }

    // X and Y with their decays (16 columns per warpgroup), as tiles over M once its last
    // reader is done.  Z = X o (Q K^T) + Y o (K K^T) below the diagonal.
    float z[16];
    {
        const Sum2 mine = gt.sum[t];
        const float sign = keys ? -1.f : a.scale;
        const int last = keys ? t - 1 : t, s0 = wg * 16;   // the last column of this row
        uint32_t g[16];
        tmem_ld16(tl + bwd_tmem::S + s0, g);
        tmem_wait_ld();
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const Sum2 o = gt.sum[s0 + i];
            const bool on = s0 + i <= last;
            x[i] = on ? __uint_as_float(g[i]) * (sign * exp2_fast(on ? (mine.hi - o.hi) + (mine.lo - o.lo) : 0.f)) : 0.f;
        }
        if (!L::BOTH) {
            ok &= tc_wait_warp(&bar.e, e_phase, gone, a.ctl);
            if (rounds == 2) add_part(bwd_tmem::C, c0);
        }
        tmem_ld16(tl + kGramAt<CT> + s0, g);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = s0 + i < t ? x[i] * __uint_as_float(g[i]) : 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            unit_terms<CT>(sm32 + L::M_AT + swizzled(tid, s0 / 8 + i), 2 * TILE, make_float4(x[8 * i], x[8 * i + 1], x[8 * i + 2], x[8 * i + 3]),
                           make_float4(x[8 * i + 4], x[8 * i + 5], x[8 * i + 6], x[8 * i + 7]));
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0 && elect_one() && ok) {
        tc_fence_after();
        // I: rows of K are the K dimension.  J: [X;Y]'s columns in rows 64 .. 127.
        issue_ss<CT, NT, CT - 1, 4>(tm + bwd_tmem::I, smem_desc(sm32 + L::M_AT, 16, 1024), 2 * TILE,
                                    smem_desc(sm32 + L::QK_AT + TILE, 2 * TILE, 1024), L::QK_TERM, mma_desc(128, DK, false, true), KMajor1(),
                                    MNMajor());
        issue_ss<CT, NT, CT - 1, 8>(tm + bwd_tmem::J, smem_desc(sm32 + L::M_AT - TILE, TILE, 1024), 2 * TILE,
                                    smem_desc(sm32 + L::QK_AT, 2 * TILE, 1024), L::QK_TERM, mma_desc(128, DK, true, true), MNMajor(), MNMajor());
        mma_commit(&bar.r);
    }
    __syncwarp();
    // Z's part of dg while the products run: dg_t gathers Z_rs for r >= t > s.  Z goes to U's
    // place (16-byte units swizzled), a thread takes eight rows of a column and adds them up from below.
    ok &= tc_wait_warp(&bar.e, e_phase, gone, a.ctl);
    {
        float *zs = reinterpret_cast<float *>(sm + L::U_AT);
        static_assert(128 * 64 * 4 <= CT * 2 * TILE, "U's place holds Z's two halves");
#pragma unroll
        for (int i = 0; i < 4; ++i) store4(zs + tid * 64 + (((wg * 4 + i) ^ (tid & 15)) << 2), make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]));
        __syncthreads();
        const int s = threadIdx.x % 64, part = threadIdx.x / 64;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int r = part * 8 + j, at = (((s >> 2) ^ (r & 15)) << 2) + (s & 3);
            v[j] = zs[r * 64 + at] + zs[(64 + r) * 64 + at];
        }
#pragma unroll
        for (int j = 6; j >= 0; --j) v[j] += v[j + 1];
        rows[row_sums::TOTAL + part * 64 + s] = v[0];
        __syncthreads();
        float below = 0.f;
        for (int q = 7; q > part; --q) below += rows[row_sums::TOTAL + q * 64 + s];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = s < part * 8 + j ? v[j] + below : 0.f;
        // The warp's 32 columns: each exchange halves the steps that a lane still holds.
#pragma unroll
        for (int n = 4, o = 16; n; n /= 2, o /= 2)
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const bool up = lane & o;
                const float give = up ? v[j] : v[j + n], keep = up ? v[j + n] : v[j];
                v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
        if (lane % 4 == 0) rows[row_sums::Z + s / 32 * 64 + part * 8 + lane / 4] = v[0];
    }
    // Eight values of this thread's row of Q or K, from x0 on.
    auto qk_row = [&](int x0, float *f) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = 0.f;
#pragma unroll
        for (int j = NT - 1; j >= 0; --j) {
            const uint4 p = *reinterpret_cast<const uint4 *>(sm + L::QK_AT + j * L::QK_TERM + (x0 / 64 * 2 + keys) * TILE + swizzled(t, x0 % 64 / 8));
            const float4 lo = IoBF16::get(make_uint2(p.x, p.y)), hi = IoBF16::get(make_uint2(p.z, p.w));
            f[0] += lo.x, f[1] += lo.y, f[2] += lo.z, f[3] += lo.w, f[4] += hi.x, f[5] += hi.y, f[6] += hi.z, f[7] += hi.w;
        }
    };
    ok &= tc_wait_warp(&bar.r, 0, gone, a.ctl);
    // dq and dk: rows to tiles in shared memory (every operand is done with), then whole lines out.
    constexpr uint32_t OUT_ROW = DK * 4 + 16;   // padded fp32 rows
    static_assert(L::U_AT + 128 * OUT_ROW <= L::GATES_AT, "the operands' place holds the rows of dq and dk");
    {
        float own = 0.f, part = 0.f;   // a's part of this row, and b's
        const float fr = keys ? -gt.grown[t] : a.scale * gt.grown[t], fc = keys ? gt.left[t] : 0.f;
#pragma unroll 1
        for (int x0 = wg * DK / 4; x0 < (wg + 1) * DK / 4; x0 += 16) {
            uint32_t r[16], i2[16], c1[16], j2[16];
            __syncwarp();
            tmem_ld16(tl + bwd_tmem::R + x0, r);
            tmem_ld16(tl + bwd_tmem::I + x0, i2);
            tmem_ld16(tl + bwd_tmem::C + x0, c1);
            tmem_ld16(tl + bwd_tmem::J + x0, j2);
            tmem_wait_ld();
            float *out = reinterpret_cast<float *>(sm + L::U_AT + tid * OUT_ROW) + x0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float f[8], v[8];
                qk_row(x0 + 8 * h, f);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float rs = fr * __uint_as_float(r[8 * h + k]), w = rs + __uint_as_float(i2[8 * h + k]);
                    float cs = 0.f, col = 0.f;   // (a query's rows of C and J hold nothing)
                    if (keys) cs = fc * __uint_as_float(c1[8 * h + k]), col = cs + __uint_as_float(j2[8 * h + k]);
                    part = fmaf(f[k], cs, part);
                    own = fmaf(f[k], rs, own);
                    v[k] = w + col;
                }
                store4(out + 8 * h, make_float4(v[0], v[1], v[2], v[3]));
                store4(out + 8 * h + 4, make_float4(v[4], v[5], v[6], v[7]));
            }
        }
        rows[row_sums::A + wg * 128 + tid] = own;
        if (keys) rows[row_sums::B + wg * 64 + t] = part;
    }
    __syncthreads();
    {
        const bool shared = a.Hv != a.Hk;
        constexpr int PER = 8, UN = DK / PER;   // values per store of a thread
#pragma unroll 2
        for (int i = threadIdx.x; i < 128 * UN; i += kChunkThreads) {
            const int r = i / UN, x = i % UN * PER, s = r % 64;
            if (s < left && x < a.Dk) {
                const float *src = reinterpret_cast<const float *>(sm + L::U_AT + r * OUT_ROW) + x;
                const float4 v[2] = {*reinterpret_cast<const float4 *>(src), *reinterpret_cast<const float4 *>(src + 4)};
                const size_t at = ((size_t)(row0 + s) * a.Hv + head) * a.Dk + x;
                if (shared) store_quads<2>((r < 64 ? a.dqh : a.dkh) + at, v);
                else store_quads<2>(static_cast<T *>(r < 64 ? a.dq : a.dk) + at, v);
            }
        }
    }
    if (warp == 0) {   // dg: a from the step on, b of the steps before it, Z's part and the state's
        float whole = lane < 16 ? rows[row_sums::MD + lane] : 0.f;
#pragma unroll
        for (int o = 16; o; o /= 2) whole += __shfl_xor_sync(0xffffffffu, whole, o);
        float d[2], b[2], from = 0.f, upto = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int s = 2 * lane + i;
            d[i] = b[i] = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) d[i] += rows[row_sums::A + 64 * w + s];
#pragma unroll
            for (int w = 0; w < 4; ++w) b[i] += rows[row_sums::B + 64 * w + s];
            from += d[i], upto += b[i];
        }
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const float right = __shfl_down_sync(0xffffffffu, from, o), earlier = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane + o < 32) from += right;
            if (lane >= o) upto += earlier;
        }
        const float next = __shfl_down_sync(0xffffffffu, from, 1), last = __shfl_up_sync(0xffffffffu, upto, 1);
        const float after = (lane < 31 ? next : 0.f) + d[1], before = lane ? last : 0.f;   // a from step 2 lane + 1 on; b before step 2 lane
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int s = 2 * lane + i;
            if (s < left)
                store_any(a.dg, a.gate16, (row0 + s) * a.Hv + head,
                          (i ? after : from) + (i ? before + b[0] : before) + (rows[row_sums::Z + s] + rows[row_sums::Z + 64 + s]) + whole);
        }
    }
    if (warp == 0 && elect_one() && (!ok || *gone)) drain_products(&bar.drain, a.ctl);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free_all(tm);
}

}  // namespace qs
