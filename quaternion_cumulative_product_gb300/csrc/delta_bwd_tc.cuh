// delta_bwd_tc.cuh -- backward of the gated delta rule on the tensor cores: the
// gradients of one chunk from the state that enters it, the cotangent of the
// state that leaves it, its errors e and its w.
//
// One CTA per (chunk, value head), four warpgroups that share the 128 rows of each
// product (each takes a quarter of the columns).  Rows of queries and of keys are
// stacked, so that one product serves both:
//
//     [dO; dV] U^T                -> X, Y (64 + 64 rows, with the decays)
//     [dO; dV] M^T                -> the states' part of dq and of row
//     [X; Y] K                    -> the rest of dq and of row
//     [Q; K]^T [X; Y]  (dk x s)   -> col, transposed
//     dM' U^T          (dk x s)   -> the state's part of col
//
// (names as in delta_common.cuh).  The stacked left operand and dM' are in tensor
// memory, the others in shared memory; [X;Y] is a K-major operand in one product and
// an MN-major one in the other.
//
// Terms: CT bfloat16 terms per computed value: three (fp32 precision) where any
// output is fp32; two (16 bits) where outputs and gates are bfloat16, whose own
// rounding is 2^-9.
#pragma once

#include "delta_prep.cuh"

namespace qs {

constexpr int kChunkThreads = 512;

template <int NT, int CT, int DK>
struct ChunkLayout {
    static constexpr int HALVES = DK / 64;
    static constexpr int MHALVES = NT == 1 ? 2 : 1;                      // halves of dv of M held at a time
    static constexpr uint32_t M_HALF = DK * 128, M_TERM = MHALVES * M_HALF;
    static constexpr int CLD = DK + 4;                                   // col [64][CLD] fp32, over U
    static constexpr uint32_t U_NEED = CT * 2 * TILE, C_NEED = (64 * CLD * 4 + 1023) / 1024 * 1024;
    static constexpr uint32_t U_AT = 0, QK_AT = U_NEED > C_NEED ? U_NEED : C_NEED;   // U: [term][half of dv][64 rows]
    static constexpr uint32_t M_AT = QK_AT + NT * HALVES * 2 * TILE;     // M: [term][half of dv][DK rows]
    static constexpr uint32_t M_BYTES = CT * M_TERM > CT * 2 * TILE ? CT * M_TERM : CT * 2 * TILE;   // then [X;Y]: [term][128 rows]
    static constexpr uint32_t GATES_AT = M_AT + M_BYTES, ROWS_AT = GATES_AT + sizeof(ChunkGates);
    static constexpr uint32_t BARS_AT = ROWS_AT + (4 * 128 + 32) * 4;
    static constexpr uint32_t NEED = BARS_AT + 256 + 1024;
    static constexpr uint32_t BYTES = NEED > 117760 ? NEED : 117760;     // one CTA per SM: it takes all of the tensor memory
    static_assert(BYTES <= 232448, "227 KB of shared memory");
};

namespace bwd_tmem {
constexpr uint32_t A = 0;      // terms (3 x 64) of [dO; dV], then of dM'
constexpr uint32_t XY = 192;   // [dO; dV] U^T (64)
constexpr uint32_t R = 256;    // dq and row (128)
constexpr uint32_t C = 384, E = 448;   // [Q;K]^T [X;Y] and dM' U^T (64 each)
}  // namespace bwd_tmem

struct ChunkBars {
    uint64_t m, xy, c, e, r;
    uint32_t tmem;
    int gone;
};

// Sixteen fp32 values of row r from value 16p into CT terms: tensor-memory columns.
template <int CT>
__device__ __forceinline__ void terms_to_tmem(uint32_t at, uint32_t term, const float *x) {
    uint32_t t[CT][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t p[3];
        split2<CT>(x[2 * i], x[2 * i + 1], p);
#pragma unroll
        for (int j = 0; j < CT; ++j) t[j][i] = p[j];
    }
#pragma unroll
    for (int j = 0; j < CT; ++j) tmem_st8(at + j * term, t[j]);
}

__device__ __forceinline__ void load16(const float *p, bool in, float *x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 v = in ? __ldg(reinterpret_cast<const float4 *>(p) + i) : q_zero();
        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16 *p, bool in, float *x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 v = in ? __ldg(reinterpret_cast<const uint4 *>(p) + i) : make_uint4(0, 0, 0, 0);
        const float4 a = IoBF16::get(make_uint2(v.x, v.y)), b = IoBF16::get(make_uint2(v.z, v.w));
        x[8 * i] = a.x, x[8 * i + 1] = a.y, x[8 * i + 2] = a.z, x[8 * i + 3] = a.w;
        x[8 * i + 4] = b.x, x[8 * i + 5] = b.y, x[8 * i + 6] = b.z, x[8 * i + 7] = b.w;
    }
}

// Sixteen values of a head row of length D from x0, as far as they exist (D is a multiple of 8).
template <typename T>
__device__ __forceinline__ void load16_upto(const T *p, bool in, int x0, int D, float *x) {
    if (x0 + 16 <= D) {
        load16(p + x0, in, x);
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 v = in && x0 + i < D ? load4(p + x0 + i) : q_zero();
            x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
        }
    }
}

template <typename T, int NT, int CT, int DK>
__global__ void __launch_bounds__(kChunkThreads, 1) delta_chunk_tc_kernel(const __grid_constant__ DeltaArgs a) {
    using L = ChunkLayout<NT, CT, DK>;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024u - smem_addr(raw) % 1024u) % 1024u);
    const uint32_t sm32 = smem_addr(sm);
    ChunkBars &bar = *reinterpret_cast<ChunkBars *>(sm + L::BARS_AT);
    ChunkGates &gt = *reinterpret_cast<ChunkGates *>(sm + L::GATES_AT);
    float *rows = reinterpret_cast<float *>(sm + L::ROWS_AT);   // [4][128] row sums, then 2 x 16 sums of the warps
    volatile int *gone = &bar.gone;

    const int head = blockIdx.x % a.Hv, kh = head / (a.Hv / a.Hk);
    Seq seq;
    long long c;
    if (!chunk_of(a, blockIdx.x / a.Hv, &seq, &c)) return;
    const long long t0 = c * DC, row0 = seq.b * a.S + seq.s0 + t0;
    const int left = (int)min((long long)DC, seq.len - t0);
    const int wg = warp_uniform(threadIdx.x / 128), tid = threadIdx.x % 128, warp = warp_uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const int t = tid % 64;
    const bool live = t < left, keys = tid >= 64;   // this thread's row: a query's or a key's
    const size_t at0 = ((size_t)(seq.slot0 + c) * a.Hv + head) * a.Dk * a.Dv;
    const float *m = a.carries_in + at0, *dm = a.ds + at0;
    const int dvp = a.Dv <= 64 ? 64 : 128, ksteps = dvp / 16;

    if (threadIdx.x == 0) {
        for (uint64_t *b : {&bar.m, &bar.xy, &bar.c, &bar.e, &bar.r}) mbar_init(b, 1);
        *gone = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc_all(&bar.tmem);
    if (warp == 1) warp_gates(gt, read_gates(a, seq, t0, head));
    {   // Q by half of the threads, K by the others
        const int w = wg / 2;
        load_rows<T, NT, DK, 256>(sm32 + L::QK_AT + w * TILE, 2 * TILE, L::HALVES * 2 * TILE, w ? a.k : a.q, w ? a.sk : a.sq, seq, t0, kh,
                                  a.Dk, threadIdx.x % 256);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = (uint32_t)warp_uniform((int)bar.tmem), tl = tm + ((uint32_t)(warp % 4 * 32) << 16);

    // M (or the first half of dv of it) into tiles: eight values per step of a thread.
    auto load_m = [&](int half0, int halves) {
        const int units = halves * 8;   // per row
#pragma unroll 4
        for (int i = threadIdx.x; i < DK * units; i += kChunkThreads) {
            const int r = i / units, u = i - r * units, x0 = half0 * 64 + u * 8;
            const bool in = r < a.Dk && x0 < a.Dv;
            const float4 p = in ? __ldg(reinterpret_cast<const float4 *>(m + (size_t)r * a.Dv + x0)) : q_zero();
            const float4 q = in ? __ldg(reinterpret_cast<const float4 *>(m + (size_t)r * a.Dv + x0 + 4)) : q_zero();
            uint32_t s[4][3];
            split2<CT>(p.x, p.y, s[0]), split2<CT>(p.z, p.w, s[1]), split2<CT>(q.x, q.y, s[2]), split2<CT>(q.z, q.w, s[3]);
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const uint32_t v[4] = {s[0][j], s[1][j], s[2][j], s[3][j]};
                st_shared16(sm32 + L::M_AT + j * L::M_TERM + (u / 8) * L::M_HALF + swizzled(r, u % 8), v);
            }
        }
    };
    // D (+)= A terms (tensor memory, K steps k0 ..) x B terms (K-major).
    auto issue_a = [&](uint32_t d, uint32_t b, uint32_t b_term, uint32_t b_half, uint32_t idesc, int k0, int k1, bool add) {
        const uint64_t base = smem_desc(b, 16, 1024);
#pragma unroll
        for (int i = CT - 1; i >= 0; --i)
#pragma unroll
            for (int j = CT - 1 - i; j >= 0; --j)
#pragma unroll 4
                for (int k = k0; k < k1; ++k) {
                    mma_ts(d, tm + bwd_tmem::A + i * 64 + k * 8, base + ((j * b_term + (k - k0) / 4 * b_half + k % 4 * 32) >> 4), idesc, add);
                    add = true;
                }
    };

    // Rows of [dO; dV] into tensor memory and of U into tiles; dbeta = <e, w>.
    {
        const size_t at = ((size_t)(row0 + t) * a.Hv + head) * a.Dv;
        const T *dop = static_cast<const T *>(a.d_o) + at;
        const float *ep = a.errors_in + at, *wp = a.w + at;
        const float be = gt.beta[t];
        float dot = 0.f;
#pragma unroll 1
        for (int x0 = wg * dvp / 4; x0 < (wg + 1) * dvp / 4; x0 += 16) {
            float x[16], e[16];
            load16_upto(ep, live, x0, a.Dv, e);
            if (keys) {
                load16_upto(wp, live, x0, a.Dv, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    dot = fmaf(x[i], e[i], dot);
                    x[i] *= be;
                }
            } else {
                load16_upto(dop, live, x0, a.Dv, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) e[i] *= be;
                const uint32_t u = sm32 + L::U_AT + x0 / 64 * TILE;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t s[4][3];
#pragma unroll
                    for (int k = 0; k < 4; ++k) split2<CT>(e[8 * i + 2 * k], e[8 * i + 2 * k + 1], s[k]);
#pragma unroll
                    for (int j = 0; j < CT; ++j) {
                        const uint32_t v[4] = {s[0][j], s[1][j], s[2][j], s[3][j]};
                        st_shared16(u + j * 2 * TILE + swizzled(t, x0 % 64 / 8 + i), v);
                    }
                }
            }
            __syncwarp();
            terms_to_tmem<CT>(tl + bwd_tmem::A + x0 / 2, 64, x);
        }
        rows[wg * 128 + tid] = dot;
    }
    load_m(0, L::MHALVES);
    cp_async_wait_all();
    tmem_wait_st();
    tc_fence_before();
    fence_proxy_async_smem();
    __syncthreads();
    const uint32_t id_dk = mma_desc(128, DK), id_s = mma_desc(128, 64);
    if (warp == 0 && elect_one()) {
        tc_fence_after();
        issue_a(tm + bwd_tmem::R, sm32 + L::M_AT, L::M_TERM, L::M_HALF, id_dk, 0, min(ksteps, 4 * L::MHALVES), false);
        mma_commit(&bar.m);
        issue_a(tm + bwd_tmem::XY, sm32 + L::U_AT, 2 * TILE, TILE, id_s, 0, ksteps, false);
        mma_commit(&bar.xy);
    }
    if (wg == 1 && !keys && live)
        store_any(a.dbeta, a.gate16, (row0 + t) * a.Hv + head,
                  (rows[64 + t] + rows[192 + t]) + (rows[320 + t] + rows[448 + t]));
    __syncwarp();
    uint32_t m_phase = 0;
    tc_wait_warp(&bar.m, m_phase, gone, a.ctl);
    if (L::MHALVES == 1 && ksteps > 4) {   // the second half of dv
        m_phase = 1;
        load_m(1, 1);
        fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0 && elect_one()) {
            tc_fence_after();
            issue_a(tm + bwd_tmem::R, sm32 + L::M_AT, L::M_TERM, L::M_HALF, id_dk, 4, 8, true);
            mma_commit(&bar.m);
        }
        __syncwarp();
        tc_wait_warp(&bar.m, m_phase, gone, a.ctl);
    }

    // X and Y with their decays into tiles over M.  Each warpgroup takes 16
    // columns.
    tc_wait_warp(&bar.xy, 0, gone, a.ctl);
    {
        const Sum2 mine = gt.sum[t];
        const float sign = keys ? -1.f : a.scale;
        const int last = keys ? t - 1 : t;   // the last column of this row
        {
            const int s0 = wg * 16;
            uint32_t g[16];
            tmem_ld16(tl + bwd_tmem::XY + s0, g);
            tmem_wait_ld();
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const Sum2 o = gt.sum[s0 + i];
                const bool on = s0 + i <= last;
                x[i] = on ? __uint_as_float(g[i]) * (sign * exp2_fast(on ? (mine.hi - o.hi) + (mine.lo - o.lo) : 0.f)) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t s[4][3];
#pragma unroll
                for (int k = 0; k < 4; ++k) split2<CT>(x[8 * i + 2 * k], x[8 * i + 2 * k + 1], s[k]);
#pragma unroll
                for (int j = 0; j < CT; ++j) {
                    const uint32_t v[4] = {s[0][j], s[1][j], s[2][j], s[3][j]};
                    st_shared16(sm32 + L::M_AT + j * 2 * TILE + swizzled(tid, s0 / 8 + i), v);
                }
            }
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    constexpr uint32_t qk_term = L::HALVES * 2 * TILE;
    if (warp == 0 && elect_one()) {   // [Q;K]^T [X;Y]: both MN-major, 128 rows of K
        tc_fence_after();
        const uint32_t id = mma_desc(128, 64, true, true);   // (rows past DK hold nothing and are not read)
        const uint64_t qk = smem_desc(sm32 + L::QK_AT, 2 * TILE, 1024), xy = smem_desc(sm32 + L::M_AT, 16, 1024);
        bool add = false;
#pragma unroll
        for (int i = NT - 1; i >= 0; --i)
#pragma unroll
            for (int j = CT - 1; j >= 0; --j) {
                if (i + j > CT - 1) continue;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    mma_ss(tm + bwd_tmem::C, qk + ((i * qk_term + k * 2048) >> 4), xy + ((j * 2 * TILE + k * 2048) >> 4), id, add);
                    add = true;
                }
            }
        mma_commit(&bar.c);
    }
    __syncwarp();
    // The states' part of dq and row gets its decay; dM' takes [dO; dV]'s place; <M, dM'>.
    {
        const float f = keys ? -gt.grown[t] : a.scale * gt.grown[t];
        const float2 f2 = make_float2(f, f);
#pragma unroll 1
        for (int x0 = wg * DK / 4; x0 < (wg + 1) * DK / 4; x0 += 16) {
            uint32_t r[16];
            tmem_ld16(tl + bwd_tmem::R + x0, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 y = mul2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), f2);
                r[2 * i] = __float_as_uint(y.x), r[2 * i + 1] = __float_as_uint(y.y);
            }
            tmem_st16(tl + bwd_tmem::R + x0, r);
        }
        float dot = 0.f;
        const bool in = tid < a.Dk;
#pragma unroll 1
        for (int x0 = wg * dvp / 4; x0 < (wg + 1) * dvp / 4; x0 += 16) {
            float x[16], y[16];
            load16_upto(dm + (size_t)tid * a.Dv, in, x0, a.Dv, x);
            load16_upto(m + (size_t)tid * a.Dv, in, x0, a.Dv, y);
#pragma unroll
            for (int i = 0; i < 16; ++i) dot = fmaf(x[i], y[i], dot);
            __syncwarp();
            terms_to_tmem<CT>(tl + bwd_tmem::A + x0 / 2, 64, x);
        }
        dot *= gt.whole;
#pragma unroll
        for (int o = 16; o; o /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) rows[512 + warp] = dot;
    }
    tmem_wait_st();
    tc_fence_before();
    __syncthreads();
    if (warp == 0 && elect_one()) {
        tc_fence_after();
        issue_a(tm + bwd_tmem::E, sm32 + L::U_AT, 2 * TILE, TILE, id_s, 0, ksteps, false);
        mma_commit(&bar.e);
        // [X;Y] K: rows of K are the K dimension
        const uint32_t id = mma_desc(128, DK, false, true);
        const uint64_t xy = smem_desc(sm32 + L::M_AT, 16, 1024), kk = smem_desc(sm32 + L::QK_AT + TILE, 2 * TILE, 1024);
#pragma unroll
        for (int i = CT - 1; i >= 0; --i)
#pragma unroll
            for (int j = NT - 1; j >= 0; --j) {
                if (i + j > CT - 1) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ss(tm + bwd_tmem::R, xy + ((i * 2 * TILE + k * 32) >> 4), kk + ((j * qk_term + k * 2048) >> 4), id, true);
            }
        mma_commit(&bar.r);
    }
    __syncwarp();

    // One value of K (from its terms) at row s, column x.
    auto qk_value = [&](int which, int s, int x) {
        float v = 0.f;
#pragma unroll
        for (int j = NT - 1; j >= 0; --j) {
            const unsigned char *p = sm + L::QK_AT + j * qk_term + (x / 64 * 2 + which) * TILE + swizzled(s, x % 64 / 8) + x % 8 * 2;
            v += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p));
        }
        return v;
    };
    // col, transposed back through shared memory over U; the sum of exp(G_C - G_t) <k_t, dM' u_t>.
    tc_wait_warp(&bar.c, 0, gone, a.ctl);
    tc_wait_warp(&bar.e, 0, gone, a.ctl);
    float *col = reinterpret_cast<float *>(sm + L::U_AT);
    {
        float part = 0.f;
        const bool in = tid < DK;
        const int s0 = wg * 16;
        uint32_t x[16], y[16];
        tmem_ld16(tl + bwd_tmem::C + s0, x);
        tmem_ld16(tl + bwd_tmem::E + s0, y);
        tmem_wait_ld();
        if (in)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float e = gt.left[s0 + i] * __uint_as_float(y[i]);
                part = fmaf(e, qk_value(1, s0 + i, tid), part);
                x[i] = __float_as_uint(__uint_as_float(x[i]) + e);
            }
#pragma unroll
        for (int o = 16; o; o /= 2) part += __shfl_xor_sync(0xffffffffu, part, o);
        if (lane == 0) rows[528 + warp] = part;
        // (U's last reader is done: bar.e.)
        if (in)
#pragma unroll
            for (int i = 0; i < 16; ++i) col[(s0 + i) * L::CLD + tid] = __uint_as_float(x[i]);
    }
    tc_wait_warp(&bar.r, 0, gone, a.ctl);
    __syncthreads();
    {
        const bool shared = a.Hv != a.Hk;
        const size_t at = ((size_t)(row0 + t) * a.Hv + head) * a.Dk;
        float sum = 0.f;
#pragma unroll 1
        for (int x0 = wg * DK / 4; x0 < (wg + 1) * DK / 4; x0 += 16) {
            uint32_t r[16];
            __syncwarp();
            tmem_ld16(tl + bwd_tmem::R + x0, r);
            tmem_wait_ld();
            float v[16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {   // <q, dq> or <k, row - col>
                float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = NT - 1; j >= 0; --j) {
                    const uint4 p = *reinterpret_cast<const uint4 *>(sm + L::QK_AT + j * qk_term + (x0 / 64 * 2 + keys) * TILE +
                                                                     swizzled(t, x0 % 64 / 8 + i));
                    const float4 lo = IoBF16::get(make_uint2(p.x, p.y)), hi = IoBF16::get(make_uint2(p.z, p.w));
                    f[0] += lo.x, f[1] += lo.y, f[2] += lo.z, f[3] += lo.w, f[4] += hi.x, f[5] += hi.y, f[6] += hi.z, f[7] += hi.w;
                }
                float cl[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (keys) {
                    const float4 lo = *reinterpret_cast<const float4 *>(col + t * L::CLD + x0 + 8 * i);
                    const float4 hi = *reinterpret_cast<const float4 *>(col + t * L::CLD + x0 + 8 * i + 4);
                    cl[0] = lo.x, cl[1] = lo.y, cl[2] = lo.z, cl[3] = lo.w, cl[4] = hi.x, cl[5] = hi.y, cl[6] = hi.z, cl[7] = hi.w;
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float w = __uint_as_float(r[8 * i + k]);
                    sum = fmaf(f[k], w - cl[k], sum);
                    v[8 * i + k] = w + cl[k];
                }
            }
            if (live) {
#pragma unroll
                for (int i = 0; i < 16; i += 8)
                    if (x0 + i < a.Dk) {
                        const float4 p[2] = {make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]), make_float4(v[i + 4], v[i + 5], v[i + 6], v[i + 7])};
                        if (shared) store_quads<2>((keys ? a.dkh : a.dqh) + at + x0 + i, p);
                        else store_quads<2>(static_cast<T *>(keys ? a.dk : a.dq) + at + x0 + i, p);
                    }
            }
        }
        rows[wg * 128 + tid] = sum;
    }
    __syncthreads();
    if (warp == 0) {   // dg: suffix sums of dG, the last step's own part included in all
        float tail = rows[512 + lane];
#pragma unroll
        for (int o = 16; o; o /= 2) tail += __shfl_xor_sync(0xffffffffu, tail, o);
        float d[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int s = 2 * lane + i;
            d[i] = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) d[i] += rows[64 * w + s];
        }
        float run = d[0] + d[1];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const float other = __shfl_down_sync(0xffffffffu, run, o);
            if (lane + o < 32) run += other;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (2 * lane + i < left)
                store_any(a.dg, a.gate16, (row0 + 2 * lane + i) * a.Hv + head, run + tail - (i ? d[0] : 0.f));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free_all(tm);
}

}  // namespace qs
