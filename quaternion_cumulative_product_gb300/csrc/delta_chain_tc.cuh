// delta_chain_tc.cuh -- backward of the gated delta rule on the tensor cores: the
// chain of the states' cotangents, from the last chunk to the first.
//
// One CTA walks the chunks of one (sequence, value head) in reverse, laid out as the
// forward walk (delta_fwd_tc.cuh): dM^T [dv][dk] in tensor memory, one value row per
// thread.  With T = (1 + diag(beta) A)^-1:
//
//     R = dO^T P              (only the chunk's own inputs: runs while dM' is converted)
//     X = dM'^T K^T
//     w = (exp(G_C - G) X + R) T
//     dM = exp(G_C) dM' + (scale exp(G) dO)^T Q - (exp(G) beta w)^T K
//
//   prep    as in the forward, one chunk ahead (K, Q, dO; T, P)
//   chain   X, w and w's part of the update; half of dM's conversion
//   out     dO's part of the update; the other half; writes w and dv
//
// T and P are read across their rows (MN-major), dO^T as an MN-major left operand.
#pragma once

#include "delta_fwd_tc.cuh"

namespace qs {

template <int NT, int DK, int STAGES>
struct ChainLayout {
    static constexpr int HALVES = DK / 64;
    static constexpr uint32_t KQ = NT * HALVES * 2 * TILE;
    static constexpr uint32_t O_AT = KQ, T_AT = O_AT + NT * 2 * TILE, P_AT = T_AT + 3 * TILE, STAGE = P_AT + 3 * TILE;   // dO: [term][half of dv]
    static constexpr uint32_t F_AT = STAGES * STAGE, Y_AT = F_AT + DC * FLD * 4;
    static constexpr uint32_t GATES_AT = Y_AT + 32 * 36 * 4;
    static constexpr uint32_t BARS_AT = GATES_AT + STAGES * sizeof(ChunkGates);
    static constexpr uint32_t BYTES = BARS_AT + 256 + 1024;
    static_assert(BYTES <= 232448, "227 KB of shared memory");
    static_assert(BYTES > 116736, "one CTA per SM: it takes all of the tensor memory");
};

namespace chain_tmem {
constexpr uint32_t M = 0;      // dM (128)
constexpr uint32_t SP = 128;   // terms of dM' (3 x 64), later of X + R, then scale exp(G) dO (3 x 32), and of exp(G) beta w (3 x 32)
constexpr uint32_t X = 320;    // X, then w
constexpr uint32_t R = 384;
constexpr uint32_t G = 448;
}  // namespace chain_tmem

template <typename T, int NT, int DK, int STAGES>
__global__ void __launch_bounds__(kWalkThreads, 1) delta_chain_tc_kernel(const __grid_constant__ DeltaArgs a) {
    using L = ChainLayout<NT, DK, STAGES>;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = raw + ((1024u - smem_addr(raw) % 1024u) % 1024u);
    const uint32_t sm32 = smem_addr(sm);
    WalkBars &bar = *reinterpret_cast<WalkBars *>(sm + L::BARS_AT);
    volatile int *gone = &bar.gone;
    ChunkGates *gates = reinterpret_cast<ChunkGates *>(sm + L::GATES_AT);

    const int head = blockIdx.x % a.Hv, kh = head / (a.Hv / a.Hk);
    const long long n = blockIdx.x / a.Hv;
    const Seq seq = seq_of(a, n);
    const int chunks = (int)((seq.len + DC - 1) / DC);
    const int wg = threadIdx.x / 128, tid = threadIdx.x % 128, warp = threadIdx.x / 32;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1 + 128);   // the products, and `out` done with beta
        }
        for (uint64_t *b : {&bar.x, &bar.e, &bar.s, &bar.g}) mbar_init(b, 1);
        *gone = 0;
        fence_mbar_init();
    }
    for (int st = 0; st < STAGES; ++st)   // T and P are zero above the diagonal blocks
        for (uint32_t i = threadIdx.x; i < 6 * TILE / 16; i += kWalkThreads) {
            const uint32_t z[4] = {0, 0, 0, 0};
            st_shared16(sm32 + st * L::STAGE + L::T_AT + i * 16, z);
        }
    if (warp == 0) tmem_alloc_all(&bar.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = bar.tmem;
    const uint32_t tl = tm + ((uint32_t)(warp % 4 * 32) << 16);   // this warp's lanes
    constexpr uint32_t kq_half = 2 * TILE, kq_term = L::HALVES * kq_half;
    const qsh::Strides so = {(long long)a.S * a.Hv * a.Dv, (long long)a.Hv * a.Dv, a.Dv};

    if (wg == 2) {
        // ------------------------------------------------------------ prep
        float *tf = reinterpret_cast<float *>(sm + L::F_AT), *yf = reinterpret_cast<float *>(sm + L::Y_AT);
        RawGates raw_gates = {};
        if (tid < 32 && chunks > 0) raw_gates = read_gates(a, seq, (long long)(chunks - 1) * DC, head);
#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            const int st = it % STAGES;
            const uint32_t stage = sm32 + st * L::STAGE;
            const long long t0 = (long long)(chunks - 1 - it) * DC;
            ChunkGates &gt = gates[st];
            tc_wait_warp(&bar.empty[st], ((it / STAGES) & 1) ^ 1, gone, a.ctl);
            load_rows<T, NT, DK>(stage, kq_half, kq_term, a.k, a.sk, seq, t0, kh, a.Dk, tid);
            load_rows<T, NT, DK>(stage + TILE, kq_half, kq_term, a.q, a.sq, seq, t0, kh, a.Dk, tid);
            load_rows<T, NT, 128>(stage + L::O_AT, TILE, 2 * TILE, a.d_o, so, seq, t0, head, a.Dv, tid);
            if (t0 > 0) {
                prefetch_rows<T>(a.k, a.sk, seq, t0 - DC, kh, a.Dk, tid);
                prefetch_rows<T>(a.q, a.sq, seq, t0 - DC, kh, a.Dk, tid);
                prefetch_rows<T>(a.d_o, so, seq, t0 - DC, head, a.Dv, tid);
            }
            if (tid < 32) {
                warp_gates(gt, raw_gates);
                if (t0 > 0) raw_gates = read_gates(a, seq, t0 - DC, head);
            }
            cp_async_wait_all();
            fence_proxy_async_smem();
            named_bar_sync(2, 128);
            if (tid == 0) {
                tc_fence_after();
                issue_gram<NT, DK>(tm + chain_tmem::G, stage);
                mma_commit(&bar.g);
            }
            __syncwarp();
            tc_wait_warp(&bar.g, it & 1, gone, a.ctl);
            gram_rows(tl + chain_tmem::G, gt, tid, [&](int s0, float *x) {
                const int t = tid % 64;
                if (tid < 64) {   // beta_t A_ts, zero on the diagonal
                    const float be = gt.beta[t];
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        float y[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) y[j] = s0 + i + j == t ? 0.f : x[i + j] * be;
                        store4(tf + t * FLD + s0 + i, make_float4(y[0], y[1], y[2], y[3]));
                    }
                } else {          // P_ts
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] *= a.scale;
                    store_terms<3>(stage + L::P_AT, t, s0 / 8, x);
                    store_terms<3>(stage + L::P_AT, t, s0 / 8 + 1, x + 8);
                }
            });
            tc_fence_before();
            named_bar_sync(2, 128);
            invert_64(tf, yf, tid, 2);
            store_inverse(stage + L::T_AT, tf, tid);
            fence_proxy_async_smem();
            named_bar_sync(2, 128);
            if (tid == 0) mbar_arrive(&bar.full[st]);
        }
    } else {
        // --------------------------------------------- chain (0) and out (1)
        constexpr int HALF = DK / 2;             // columns of dM per thread
        const int dv = tid, col0 = wg * HALF;
        const bool in = dv < a.Dv;
        const size_t state = ((size_t)n * a.Hv + head) * a.Dk * a.Dv + dv;
        auto k_major = [](int k) { return (uint32_t)((k / 4) * 2 * TILE + (k % 4) * 32); };   // K [t][dk]: K steps along dk
        auto mn_major = [](int k) { return (uint32_t)(k * 2048); };                          // K, Q, T, P: K steps along the rows
        const long long row0 = seq.b * a.S + seq.s0;

#pragma unroll 1
        for (int h = 0; h < HALF; h += 16) {
            uint32_t r[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                r[i] = __float_as_uint(a.d_final && in && col0 + h + i < a.Dk ? __ldg(a.d_final + state + (size_t)(col0 + h + i) * a.Dv) : 0.f);
            __syncwarp();
            tmem_st16(tl + chain_tmem::M + col0 + h, r);
        }
        tmem_wait_st();

#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            const int st = it % STAGES, c = chunks - 1 - it;
            const uint32_t stage = sm32 + st * L::STAGE;
            const ChunkGates &gt = gates[st];
            const int left = (int)min((long long)DC, seq.len - (long long)c * DC);
            tc_wait_warp(&bar.full[st], (it / STAGES) & 1, gone, a.ctl);
            if (threadIdx.x == 0) {   // R = dO^T P
                tc_fence_after();
                const uint32_t id = mma_desc(128, 64, true, true);
                const uint64_t dd = smem_desc(stage + L::O_AT, TILE, 1024), pp = smem_desc(stage + L::P_AT, 16, 1024);
                bool add = false;
#pragma unroll
                for (int i = NT - 1; i >= 0; --i)
#pragma unroll
                    for (int j = 2 - i; j >= 0; --j)
#pragma unroll
                        for (int k = 0; k < DC / 16; ++k) {
                            mma_ss(tm + chain_tmem::R, dd + ((i * 2 * TILE + k * 2048) >> 4), pp + ((j * TILE + k * 2048) >> 4), id, add);
                            add = true;
                        }
            }
            __syncwarp();
            if (it > 0) tc_wait_warp(&bar.s, (it - 1) & 1, gone, a.ctl);
            float *ds = a.ds + ((size_t)(seq.slot0 + c) * a.Hv + head) * a.Dk * a.Dv + dv;
#pragma unroll 1
            for (int h = 0; h < HALF; h += 32) {   // dM': terms, written out, and scaled for its update
                uint32_t r[32], t[3][16];
                tmem_ld32(tl + chain_tmem::M + col0 + h, r);
                tmem_wait_ld();
                const float2 w = make_float2(gt.whole, gt.whole);
                if (in) {
                    float *out = ds + (size_t)(col0 + h) * a.Dv;
#pragma unroll
                    for (int i = 0; i < 32; ++i, out += a.Dv)
                        if (col0 + h + i < a.Dk) *out = __uint_as_float(r[i]);
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 x = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                    uint32_t p[3];
                    split2<3>(x, p);
                    t[0][i] = p[0], t[1][i] = p[1], t[2][i] = p[2];
                    const float2 y = mul2(x, w);
                    r[2 * i] = __float_as_uint(y.x), r[2 * i + 1] = __float_as_uint(y.y);
                }
#pragma unroll
                for (int j = 0; j < 3; ++j) tmem_st16(tl + chain_tmem::SP + j * 64 + (col0 + h) / 2, t[j]);
                tmem_st32(tl + chain_tmem::M + col0 + h, r);
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, 256);
            if (wg == 0) {
                if (tid == 0) {
                    tc_fence_after();
                    issue_ts<3, NT, 2, DK>(tm + chain_tmem::X, [&](int i, int k) { return tm + chain_tmem::SP + i * 64 + k * 8; }, stage,
                                           kq_term, 16, mma_desc(128, 64), k_major);
                    mma_commit(&bar.x);
                }
                __syncwarp();
                tc_wait_warp(&bar.x, it & 1, gone, a.ctl);
#pragma unroll 1
                for (int h = 0; h < DC; h += 16) {
                    uint32_t r[16], y[16], t[3][8];
                    tmem_ld16(tl + chain_tmem::X + h, r);
                    tmem_ld16(tl + chain_tmem::R + h, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 l = *reinterpret_cast<const float2 *>(&gt.left[h + 2 * i]);
                        uint32_t p[3];
                        split2<3>(fma2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), l,
                                       make_float2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]))), p);
                        t[0][i] = p[0], t[1][i] = p[1], t[2][i] = p[2];
                    }
#pragma unroll
                    for (int j = 0; j < 3; ++j) tmem_st8(tl + chain_tmem::SP + j * 32 + h / 2, t[j]);
                }
                tmem_wait_st();
                tc_fence_before();
                named_bar_sync(3, 128);
                if (tid == 0) {
                    tc_fence_after();
                    issue_ts<3, 3, 2, DC>(tm + chain_tmem::X, [&](int i, int k) { return tm + chain_tmem::SP + i * 32 + k * 8; },
                                          stage + L::T_AT, TILE, 16, mma_desc(128, 64, false, true), mn_major);
                    mma_commit(&bar.e);
                }
                __syncwarp();
                tc_wait_warp(&bar.e, it & 1, gone, a.ctl);
#pragma unroll 1
                for (int h = 0; h < DC; h += 32) {   // -exp(G) beta w
                    uint32_t r[32], t[3][16];
                    tmem_ld32(tl + chain_tmem::X + h, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 g = *reinterpret_cast<const float2 *>(&gt.grown[h + 2 * i]);
                        const float2 be = *reinterpret_cast<const float2 *>(&gt.beta[h + 2 * i]);
                        uint32_t p[3];
                        split2<3>(mul2(mul2(make_float2(-__uint_as_float(r[2 * i]), -__uint_as_float(r[2 * i + 1])), be), g), p);
                        t[0][i] = p[0], t[1][i] = p[1], t[2][i] = p[2];
                    }
#pragma unroll
                    for (int j = 0; j < 3; ++j) tmem_st16(tl + chain_tmem::SP + 96 + j * 32 + h / 2, t[j]);
                }
            } else {
                tc_wait_warp(&bar.e, it & 1, gone, a.ctl);   // the terms of X + R give way to scale exp(G) dO
                const unsigned char *od = sm + st * L::STAGE + L::O_AT + dv / 64 * TILE + dv % 8 * 2;
                const uint32_t unit = (uint32_t)(dv % 64 / 8) << 4;
#pragma unroll 1
                for (int h = 0; h < DC; h += 16) {
                    uint32_t t[3][8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float v[2] = {0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int j = NT - 1; j >= 0; --j)
                                v[k] += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(
                                    od + j * 2 * TILE + (h + 2 * i + k) * 128 + (unit ^ (uint32_t)((2 * i + k) % 8 << 4))));
                        const float2 g = *reinterpret_cast<const float2 *>(&gt.grown[h + 2 * i]);
                        uint32_t p[3];
                        split2<3>(mul2(mul2(make_float2(v[0], v[1]), g), make_float2(a.scale, a.scale)), p);
                        t[0][i] = p[0], t[1][i] = p[1], t[2][i] = p[2];
                    }
#pragma unroll
                    for (int j = 0; j < 3; ++j) tmem_st8(tl + chain_tmem::SP + j * 32 + h / 2, t[j]);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, 256);
            if (threadIdx.x == 0) {
                tc_fence_after();
                const uint32_t id = mma_desc(128, DK, false, true);
                issue_ts<3, NT, 2, DC>(tm + chain_tmem::M, [&](int i, int k) { return tm + chain_tmem::SP + i * 32 + k * 8; }, stage + TILE,
                                       kq_term, kq_half, id, mn_major, true);
                issue_ts<3, NT, 2, DC>(tm + chain_tmem::M, [&](int i, int k) { return tm + chain_tmem::SP + 96 + i * 32 + k * 8; }, stage,
                                       kq_term, kq_half, id, mn_major, true);
                mma_commit(&bar.s);
                mma_commit(&bar.empty[st]);
            }
            __syncwarp();
            if (wg == 1) {   // w and dv
                const size_t step = (size_t)a.Hv * a.Dv, at = ((size_t)(row0 + (long long)c * DC) * a.Hv + head) * a.Dv + dv;
#pragma unroll 1
                for (int h = 0; h < DC; h += 32) {
                    uint32_t r[32];
                    tmem_ld32(tl + chain_tmem::X + h, r);
                    tmem_wait_ld();
                    float *wo = a.w + at + h * step;
                    T *vo = static_cast<T *>(a.dv) + at + h * step;
                    if (in)
#pragma unroll
                        for (int i = 0; i < 32; ++i, wo += step, vo += step)
                            if (h + i < left) {
                                *wo = __uint_as_float(r[i]);
                                store1(vo, gt.beta[h + i] * __uint_as_float(r[i]));
                            }
                    __syncwarp();
                }
                tc_fence_before();
                mbar_arrive(&bar.empty[st]);
            }
        }
        if (chunks > 0) tc_wait_warp(&bar.s, (chunks - 1) & 1, gone, a.ctl);
        if (a.d_init)
#pragma unroll 1
            for (int h = 0; h < HALF; h += 16) {
                uint32_t r[16];
                __syncwarp();
                tmem_ld16(tl + chain_tmem::M + col0 + h, r);
                tmem_wait_ld();
                if (in)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (col0 + h + i < a.Dk) a.d_init[state + (size_t)(col0 + h + i) * a.Dv] = __uint_as_float(r[i]);
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free_all(tm);
}

}  // namespace qs
