// delta_fwd_tc.cuh -- forward of the gated delta rule on the tensor cores.
//
// One CTA walks the chunks of one (sequence, value head).  Everything that the
// chain of states goes through is laid out transposed: the state M^T [dv][dk], the
// errors e^T [dv][t] and so on have one value row dv per tensor-memory lane, so
// one thread owns one row of every product of the chain, and no value crosses
// threads between two of them.  Three warpgroups:
//
//   prep    one chunk ahead: loads K and Q, the decays, Gram products [K;Q] K^T,
//           T = (1 + A diag(beta))^-1 (32 x 32 blocks by substitution, the corner as
//           -T22 A21 T11), and writes T and P as operands;
//   chain   X = M^T K^T;  e = (v - exp(G) X) T^T;  dM = (beta left e)^T K
//   out     Y = M^T Q^T;  o = exp(G) Y + U P^T; and half of the state's columns
//
// The state itself stays in the registers of `chain` and `out` (64 columns of
// dk each); its bfloat16 terms go to tensor memory as the next left operand.
//
// Bound: the chain's latency.  Per chunk of 64 steps and D = 128 it runs 2.1 + 1
// + 2.1 MFLOP three products after each other, each in 3 to 6 passes, with the
// conversions to terms between them; the tensor cores are busy for about three
// quarters of that.
#pragma once

#include <type_traits>

#include "delta_common.cuh"
#include "tensor_core.cuh"

namespace qs {

// Gates of one chunk in shared memory.
struct ChunkGates {
    Sum2 sum[DC];
    float beta[DC], grown[DC], left[DC];   // beta_t, exp(G_t), exp(G_C - G_t)
    float whole;                           // exp(G_C)
};

// One warp fills the gates of the chunk that starts at step t0 of the sequence.
__device__ __forceinline__ void warp_gates(ChunkGates &s, const DeltaArgs &a, const Seq &seq, long long t0, int head) {
    const int lane = threadIdx.x % 32;
    float g[2], be[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const long long t = t0 + 2 * lane + i;
        const long long at = (seq.b * a.S + seq.s0 + t) * a.Hv + head;
        g[i] = t < seq.len ? clamp_gate(load_any(a.g, a.gate16, at)) : 0.f;
        be[i] = t < seq.len ? load_any(a.beta, a.gate16, at) : 0.f;
    }
    Sum2 s0, s1;
    chunk_sums(g[0], g[1], &s0, &s1);
    const Sum2 end = {__shfl_sync(0xffffffffu, s1.hi, 31), __shfl_sync(0xffffffffu, s1.lo, 31)};
    const int t = 2 * lane;
    s.sum[t] = s0, s.sum[t + 1] = s1;
    s.beta[t] = be[0], s.beta[t + 1] = be[1];
    s.grown[t] = expf(s0.hi + s0.lo), s.grown[t + 1] = expf(s1.hi + s1.lo);
    s.left[t] = decay(end, s0), s.left[t + 1] = decay(end, s1);
    if (lane == 31) s.whole = s.grown[63];
}

// Shared memory of the walks.  A tile is 64 rows x 64 values of bfloat16 (8 KB).
// K and Q of a stage: [term][half of D]{K tile, Q tile}.
constexpr uint32_t TILE = 8192;
constexpr int FLD = 68;   // padded rows of the fp32 64 x 64 scratch (16-byte aligned)

template <int NT, int DK, int STAGES>
struct WalkLayout {
    static constexpr int HALVES = DK / 64;
    static constexpr uint32_t KQ = NT * HALVES * 2 * TILE;   // bytes of K and Q
    static constexpr int PT = NT == 1 ? 2 : 3;               // terms of P and U (o's precision)
    static constexpr uint32_t T_AT = KQ, P_AT = T_AT + 3 * TILE, STAGE = P_AT + 3 * TILE;
    static constexpr uint32_t A_AT = STAGES * STAGE, F_AT = A_AT + DC * FLD * 4, Y_AT = F_AT + DC * FLD * 4;
    static constexpr uint32_t GATES_AT = Y_AT + 32 * 36 * 4;
    static constexpr uint32_t BARS_AT = GATES_AT + STAGES * ((sizeof(ChunkGates) + 15) / 16 * 16);
    static constexpr uint32_t BYTES = BARS_AT + 256 + 1024;   // + alignment of the tiles to 1024 bytes
};

// Rows of one head into a stage's tiles as bfloat16 terms (`which`: 0 K, 1 Q);
// zeros past the sequence and past D.  bfloat16 rows are copied asynchronously.
template <typename T, int NT, int DK, int THREADS>
__device__ __forceinline__ void load_rows(uint32_t stage, int which, const void *p, const qsh::Strides &st, const Seq &seq,
                                          long long t0, int head, int D, int tid) {
    constexpr int UNITS = DK / 8;   // 16-byte units of bfloat16 in a row
    const T *base = static_cast<const T *>(p) + seq.b * st.b + (seq.s0 + t0) * st.s + (long long)head * st.h;
#pragma unroll
    for (int i = tid; i < DC * UNITS; i += THREADS) {
        const int r = i / UNITS, u = i % UNITS;
        const bool in = t0 + r < seq.len && u * 8 < D;
        const T *src = in ? base + (long long)r * st.s + u * 8 : base;
        const uint32_t at = stage + (uint32_t)((u / 8) * 2 + which) * TILE + swizzled(r, u % 8);
        if constexpr (NT == 1) {
            cp_async16_or_zero(at, in ? src : static_cast<const T *>(p), in);
        } else {
            float4 x = q_zero(), y = q_zero();
            if (in) x = load4(src), y = load4(src + 4);
            uint32_t t[4][3];
            split2<3>(x.x, x.y, t[0]), split2<3>(x.z, x.w, t[1]), split2<3>(y.x, y.y, t[2]), split2<3>(y.z, y.w, t[3]);
#pragma unroll
            for (int j = 0; j < 3; ++j)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + j * (DK / 64) * 2 * TILE), "r"(t[0][j]),
                             "r"(t[1][j]), "r"(t[2][j]), "r"(t[3][j])
                             : "memory");
        }
    }
}

__device__ __forceinline__ void st_shared16(uint32_t at, const uint32_t *v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Eight consecutive values of row r, from value 8u, as TERMS tiles TILE apart.
template <int TERMS>
__device__ __forceinline__ void store_terms(uint32_t tiles, int r, int u, const float *x) {
    uint32_t t[4][3];
#pragma unroll
    for (int i = 0; i < 4; ++i) split2<TERMS>(x[2 * i], x[2 * i + 1], t[i]);
#pragma unroll
    for (int j = 0; j < TERMS; ++j) {
        const uint32_t v[4] = {t[0][j], t[1][j], t[2][j], t[3][j]};
        st_shared16(tiles + j * TILE + swizzled(r, u), v);
    }
}

// tf = (1 + af)^-1 for the strictly lower triangular af [64][FLD]; 128 threads
// (barrier `bar`).  yf: 32 x 36 of scratch.
__device__ __forceinline__ void invert_64(const float *af, float *tf, float *yf, int tid, int bar) {
    const int blk = tid / 32, j = tid % 32;
    if (blk < 2) {   // a diagonal block per warp, a column per thread, by substitution
        const float *a = af + blk * 32 * (FLD + 1);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            float s0 = i == j ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int m = 0; m < (i + 3) / 4 * 4; m += 4) {
                const float4 r = *reinterpret_cast<const float4 *>(a + i * FLD + m);
                if (m < i) s0 = fmaf(-r.x, x[m], s0);
                if (m + 1 < i) s1 = fmaf(-r.y, x[m + 1], s1);
                if (m + 2 < i) s0 = fmaf(-r.z, x[m + 2], s0);
                if (m + 3 < i) s1 = fmaf(-r.w, x[m + 3], s1);
            }
            x[i] = s0 + s1;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) tf[(blk * 32 + i) * FLD + blk * 32 + j] = x[i];
    } else {   // the upper corner is zero
        for (int i = tid - 64; i < 32 * 8; i += 64) *reinterpret_cast<float4 *>(tf + i / 8 * FLD + 32 + i % 8 * 4) = q_zero();
    }
    named_bar_sync(bar, 128);
    const int r = tid / 8 * 2, c = tid % 8 * 4;   // a 2 x 4 piece of the corner per thread
    auto corner = [&](const float *a, const float *b, int ldb, float4 *out) {
        out[0] = out[1] = q_zero();
#pragma unroll
        for (int m = 0; m < 32; m += 4) {
            const float4 p = *reinterpret_cast<const float4 *>(a + r * FLD + m);
            const float4 q = *reinterpret_cast<const float4 *>(a + (r + 1) * FLD + m);
            const float pp[4] = {p.x, p.y, p.z, p.w}, qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 y = *reinterpret_cast<const float4 *>(b + (m + k) * ldb + c);
                out[0] = make_float4(fmaf(pp[k], y.x, out[0].x), fmaf(pp[k], y.y, out[0].y), fmaf(pp[k], y.z, out[0].z), fmaf(pp[k], y.w, out[0].w));
                out[1] = make_float4(fmaf(qq[k], y.x, out[1].x), fmaf(qq[k], y.y, out[1].y), fmaf(qq[k], y.z, out[1].z), fmaf(qq[k], y.w, out[1].w));
            }
        }
    };
    float4 y[2];
    corner(af + 32 * FLD, tf, FLD, y);
    store4(yf + r * 36 + c, y[0]);
    store4(yf + (r + 1) * 36 + c, y[1]);
    named_bar_sync(bar, 128);
    corner(tf + 32 * FLD + 32, yf, 36, y);
    store4(tf + (32 + r) * FLD + c, make_float4(-y[0].x, -y[0].y, -y[0].z, -y[0].w));
    store4(tf + (33 + r) * FLD + c, make_float4(-y[1].x, -y[1].y, -y[1].z, -y[1].w));
    named_bar_sync(bar, 128);
}

// Issues D[128 x N] (+)= sum over term pairs of A[tmem] B[smem], K values of K.
// A's terms are `a_term` columns apart, B's `b_term` bytes; `b_at(k16)` gives the
// byte offset of K step k16; pairs i + j <= LAST, i < TA, j < TB.
template <int TA, int TB, int LAST, int K, typename F>
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a, uint32_t a_term, uint32_t b, uint32_t b_term, uint32_t lbo,
                                         uint32_t idesc, const F &b_at, bool add = false) {
#pragma unroll
    for (int i = TA - 1; i >= 0; --i)   // small terms first
#pragma unroll
        for (int j = TB - 1; j >= 0; --j) {
            if (i + j > LAST) continue;
#pragma unroll
            for (int k = 0; k < K / 16; ++k) {
                mma_ts(d, a + i * a_term + k * 8, smem_desc(b + j * b_term + b_at(k), lbo, 1024), idesc, add);
                add = true;
            }
        }
}

// Tensor-memory columns of the forward walk.  With bfloat16 inputs (two terms
// for o) the operands are placed so that Y and U P^T run while the chain converts:
// the terms of v - exp(G) X take the place of M's third term, which only X needs,
// and U that of e.  With fp32 inputs Y needs all of M's terms, and the chain waits.
namespace fwd_tmem {
constexpr uint32_t D = 0;      // dM (128), then Y (64)
constexpr uint32_t SP = 128;   // terms of M (3 x 64), later of beta left e (3 x 32)
constexpr uint32_t X = 320;    // X, then e, then (bfloat16) U
constexpr uint32_t O = 384;    // U P^T
constexpr uint32_t G = 448;    // Gram products
}  // namespace fwd_tmem

constexpr int kWalkThreads = 384;

template <typename T, int NT, int DK, int STAGES>
__global__ void __launch_bounds__(kWalkThreads, 1) delta_fwd_tc_kernel(const __grid_constant__ DeltaArgs a) {
    using L = WalkLayout<NT, DK, STAGES>;
    extern __shared__ unsigned char raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sm32 = smem_addr(sm);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS_AT);
    uint64_t *full = bars, *empty = bars + 2, *bx = bars + 4, *by = bars + 5, *be = bars + 6, *bs = bars + 7, *bo = bars + 8,
             *bg = bars + 9, *yread = bars + 10, *oread = bars + 11;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 12);
    volatile int *gone = reinterpret_cast<volatile int *>(bars + 13);
    auto gates_of = [&](int st) -> ChunkGates & {
        return *reinterpret_cast<ChunkGates *>(sm + L::GATES_AT + st * ((sizeof(ChunkGates) + 15) / 16 * 16));
    };

    const int head = blockIdx.x % a.Hv, kh = head / (a.Hv / a.Hk);
    const long long n = blockIdx.x / a.Hv;
    const Seq seq = seq_of(a, n);
    const int chunks = (int)((seq.len + DC - 1) / DC);
    const int wg = threadIdx.x / 128, tid = threadIdx.x % 128, warp = threadIdx.x / 32;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (uint64_t *b : {bx, by, be, bs, bo, bg}) mbar_init(b, 1);
        mbar_init(yread, 128);
        mbar_init(oread, 128);
        *gone = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc_all(tmem_slot);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tmem_slot;
    const uint32_t lane_base = (uint32_t)(warp % 4 * 32) << 16;

    if (wg == 2) {
        // ------------------------------------------------------------ prep
        float *af = reinterpret_cast<float *>(sm + L::A_AT), *tf = reinterpret_cast<float *>(sm + L::F_AT);
        float *yf = reinterpret_cast<float *>(sm + L::Y_AT);
        for (int c = 0; c < chunks; ++c) {
            const int st = c % STAGES;
            const uint32_t stage = sm32 + st * L::STAGE;
            ChunkGates &gt = gates_of(st);
            tc_wait_warp(empty + st, ((c / STAGES) & 1) ^ 1, gone, a.ctl);
            load_rows<T, NT, DK, 128>(stage, 0, a.k, a.sk, seq, (long long)c * DC, kh, a.Dk, tid);
            load_rows<T, NT, DK, 128>(stage, 1, a.q, a.sq, seq, (long long)c * DC, kh, a.Dk, tid);
            if (tid < 32) warp_gates(gt, a, seq, (long long)c * DC, head);
            if (NT == 1) cp_async_wait_all();
            fence_proxy_async_smem();
            named_bar_sync(2, 128);
            if (tid == 0) {   // Gram: rows 0-63 K K^T, rows 64-127 Q K^T
                tc_fence_after();
                constexpr uint32_t id = mma_desc(128, 64);
                bool add = false;
#pragma unroll
                for (int i = NT - 1; i >= 0; --i)
#pragma unroll
                    for (int j = NT - 1; j >= 0; --j) {
                        if (i + j > 2) continue;
#pragma unroll
                        for (int k = 0; k < DK / 16; ++k) {
                            const uint32_t at = (k / 4) * 2 * TILE + (k % 4) * 32;
                            mma_ss(tm + fwd_tmem::G, smem_desc(stage + i * (DK / 64) * 2 * TILE + at, 16, 1024),
                                   smem_desc(stage + j * (DK / 64) * 2 * TILE + at, 16, 1024), id, add);
                            add = true;
                        }
                    }
                mma_commit(bg);
            }
            __syncwarp();
            tc_wait_warp(bg, c & 1, gone, a.ctl);
            const int t = tid % 64;
            const Sum2 mine = gt.sum[t];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t g[32];
                tmem_ld32(tm + fwd_tmem::G + lane_base + h * 32, g);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int s = h * 32 + u * 8 + i;
                        x[i] = s <= t ? decay(mine, gt.sum[s]) * __uint_as_float(g[u * 8 + i]) : 0.f;
                    }
                    if (tid < 64) {   // A_ts beta_s
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int s = h * 32 + u * 8 + i;
                            af[t * FLD + s] = s < t ? x[i] * gt.beta[s] : 0.f;
                        }
                    } else {          // P_ts
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] *= a.scale;
                        store_terms<L::PT>(stage + L::P_AT, t, h * 4 + u, x);
                    }
                }
            }
            tc_fence_before();
            named_bar_sync(2, 128);
            invert_64(af, tf, yf, tid, 2);
#pragma unroll
            for (int u = 0; u < 4; ++u) {   // half a row of T per thread
                const int r = tid / 2, uu = (tid & 1) * 4 + u;
                float x[8];
                const float4 p = *reinterpret_cast<const float4 *>(tf + r * FLD + uu * 8);
                const float4 q = *reinterpret_cast<const float4 *>(tf + r * FLD + uu * 8 + 4);
                x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w, x[4] = q.x, x[5] = q.y, x[6] = q.z, x[7] = q.w;
                store_terms<3>(stage + L::T_AT, r, uu, x);
            }
            fence_proxy_async_smem();
            named_bar_sync(2, 128);
            if (tid == 0) mbar_arrive(full + st);
        }
    } else {
        // --------------------------------------------- chain (0) and out (1)
        constexpr int HALF = DK / 2;             // columns of the state per thread
        constexpr bool kEarly = NT == 1;
        const int dv = tid, col0 = wg * HALF;
        const bool in = dv < a.Dv;
        const size_t state = ((size_t)n * a.Hv + head) * a.Dk * a.Dv;
        float m[HALF], y[DC];                    // state; Y of the chunk before (out)
        float whole = 0.f;
#pragma unroll
        for (int i = 0; i < HALF; ++i)
            m[i] = a.init && in && col0 + i < a.Dk ? __ldg(a.init + state + (size_t)(col0 + i) * a.Dv + dv) : 0.f;
        constexpr uint32_t kq_half = 2 * TILE;
        auto k_major = [](int k) { return (uint32_t)((k / 4) * 2 * TILE + (k % 4) * 32); };   // K or Q [t][dk]: K steps along dk
        auto mn_major = [](int k) { return (uint32_t)(k * 2048); };                          // K [t][dk]: K steps along t
        auto tile_k = [](int k) { return (uint32_t)(k * 32); };                              // T or P
        const T *vbase = static_cast<const T *>(a.v) + seq.b * a.sv.b + seq.s0 * a.sv.s + (long long)head * a.sv.h + dv;
        const long long row0 = seq.b * a.S + seq.s0;

        // dM of chunk c is ready: the state that enters chunk c + 1.
        auto advance = [&](int c) {
            tc_wait_warp(bs, c & 1, gone, a.ctl);
#pragma unroll
            for (int h = 0; h < HALF / 32; ++h) {
                uint32_t r[32];
                tmem_ld32(tm + fwd_tmem::D + lane_base + col0 + h * 32, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) m[h * 32 + i] = fmaf(whole, m[h * 32 + i], __uint_as_float(r[i]));
            }
        };
        // o of chunk c from Y (registers) and U P^T.
        auto write_o = [&](int c) {
            tc_wait_warp(bo, c & 1, gone, a.ctl);
            const long long left = seq.len - (long long)c * DC;
            T *out = static_cast<T *>(a.o) + ((size_t)(row0 + (long long)c * DC) * a.Hv + head) * a.Dv + dv;
            uint32_t r[DC];
            tmem_ld32(tm + fwd_tmem::O + lane_base, r);
            tmem_ld32(tm + fwd_tmem::O + lane_base + 32, r + 32);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(oread);
#pragma unroll
            for (int t = 0; t < DC; ++t)
                if (in && t < left) store1(out + (size_t)t * a.Hv * a.Dv, y[t] + __uint_as_float(r[t]));
            __syncwarp();
        };
        // TERMS bfloat16 terms of 64 values into tensor memory, term j at at(j).
        auto put_terms = [&](auto terms, const float *x, auto at) {
            constexpr int TERMS = decltype(terms)::value;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t t[TERMS][8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t p[3];
                    split2<TERMS>(x[h * 16 + 2 * i], x[h * 16 + 2 * i + 1], p);
#pragma unroll
                    for (int j = 0; j < TERMS; ++j) t[j][i] = p[j];
                }
#pragma unroll
                for (int j = 0; j < TERMS; ++j) tmem_st8(tm + lane_base + at(j) + h * 8, t[j]);
            }
        };
        using Three = std::integral_constant<int, 3>;
        using OTerms = std::integral_constant<int, L::PT>;

        for (int c = 0; c < chunks; ++c) {
            const int st = c % STAGES;
            const uint32_t stage = sm32 + st * L::STAGE;
            const ChunkGates &gt = gates_of(st);
            const long long left = seq.len - (long long)c * DC;
            if (c > 0) advance(c - 1);
            if (a.carries && in) {
                float *out = a.carries + ((size_t)(seq.slot0 + c) * a.Hv + head) * a.Dk * a.Dv + dv;
#pragma unroll
                for (int i = 0; i < HALF; ++i)
                    if (col0 + i < a.Dk) out[(size_t)(col0 + i) * a.Dv] = m[i];
            }
            __syncwarp();
            if (!kEarly && c > 0) tc_wait_warp(bo, (c - 1) & 1, gone, a.ctl);   // U lies where M's terms go
#pragma unroll
            for (int h = 0; h < HALF / 32; ++h) {
                uint32_t t[3][16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    uint32_t x[3];
                    split2<3>(m[h * 32 + 2 * i], m[h * 32 + 2 * i + 1], x);
                    t[0][i] = x[0], t[1][i] = x[1], t[2][i] = x[2];
                }
#pragma unroll
                for (int j = 0; j < 3; ++j) tmem_st16(tm + fwd_tmem::SP + lane_base + j * 64 + (col0 + h * 32) / 2, t[j]);
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, 256);
            tc_wait_warp(full + st, (c / STAGES) & 1, gone, a.ctl);
            auto issue_y = [&] {
                issue_ts<L::PT, NT, L::PT - 1, DK>(tm + fwd_tmem::D, tm + fwd_tmem::SP, 64, stage + TILE, L::HALVES * kq_half, 16,
                                                   mma_desc(128, 64), k_major);
                mma_commit(by);
            };
            whole = gt.whole;
            if (wg == 0) {
                if (tid == 0) {
                    issue_ts<3, NT, 2, DK>(tm + fwd_tmem::X, tm + fwd_tmem::SP, 64, stage, L::HALVES * kq_half, 16,
                                           mma_desc(128, 64), k_major);
                    mma_commit(bx);
                    if (!kEarly) issue_y();
                }
                float e[DC];
                {   // the values are under way while the products run
                    const T *vp = vbase + (long long)c * DC * a.sv.s;
#pragma unroll
                    for (int t = 0; t < DC; ++t) e[t] = in && t < left ? load1(vp + (long long)t * a.sv.s) : 0.f;
                }
                tc_wait_warp(bx, c & 1, gone, a.ctl);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[32];
                    tmem_ld32(tm + fwd_tmem::X + lane_base + h * 32, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) e[h * 32 + i] = fmaf(-gt.grown[h * 32 + i], __uint_as_float(r[i]), e[h * 32 + i]);
                }
                // Terms of v - exp(G) X: over M's third term and O (read by now), or
                // over M's terms once Y is done.
                if (kEarly) {
                    if (c > 0) tc_wait_warp(oread, (c - 1) & 1, gone, a.ctl);
                    put_terms(Three(), e, [](int j) { return j < 2 ? fwd_tmem::SP + 128 + j * 32 : fwd_tmem::O; });
                } else {
                    tc_wait_warp(by, c & 1, gone, a.ctl);
                    put_terms(Three(), e, [](int j) { return fwd_tmem::SP + j * 32; });
                }
                tmem_wait_st();
                tc_fence_before();
                named_bar_sync(3, 128);
                if (tid == 0) {
                    tc_fence_after();
                    constexpr uint32_t id = mma_desc(128, 64);
                    const uint32_t tt = stage + L::T_AT;
                    bool add = false;
#pragma unroll
                    for (int i = 2; i >= 0; --i) {
                        const uint32_t at = tm + (!kEarly ? fwd_tmem::SP + i * 32 : i < 2 ? fwd_tmem::SP + 128 + i * 32 : fwd_tmem::O);
#pragma unroll
                        for (int j = 2 - i; j >= 0; --j)
#pragma unroll
                            for (int k = 0; k < DC / 16; ++k) {
                                mma_ts(tm + fwd_tmem::X, at + k * 8, smem_desc(tt + j * TILE + k * 32, 16, 1024), id, add);
                                add = true;
                            }
                    }
                    mma_commit(be);
                    if (kEarly) issue_y();
                }
                tc_wait_warp(be, c & 1, gone, a.ctl);
                float *eo = a.errors ? a.errors + ((size_t)(row0 + (long long)c * DC) * a.Hv + head) * a.Dv + dv : nullptr;
                {
                    uint32_t r[DC];
                    tmem_ld32(tm + fwd_tmem::X + lane_base, r);
                    tmem_ld32(tm + fwd_tmem::X + lane_base + 32, r + 32);
                    tmem_wait_ld();
#pragma unroll
                    for (int t = 0; t < DC; ++t) e[t] = __uint_as_float(r[t]);
                }
                if (eo && in)
#pragma unroll
                    for (int t = 0; t < DC; ++t)
                        if (t < left) eo[(size_t)t * a.Hv * a.Dv] = e[t];
                __syncwarp();
#pragma unroll
                for (int t = 0; t < DC; ++t) e[t] *= gt.beta[t];
                constexpr uint32_t u_at = kEarly ? fwd_tmem::X : fwd_tmem::SP + 96;
                put_terms(OTerms(), e, [](int j) { return u_at + j * 32; });
#pragma unroll
                for (int t = 0; t < DC; ++t) e[t] *= gt.left[t];
                if (kEarly) tc_wait_warp(by, c & 1, gone, a.ctl);   // Y reads M's first terms
                put_terms(Three(), e, [](int j) { return fwd_tmem::SP + j * 32; });
                tmem_wait_st();
                tc_fence_before();
                named_bar_sync(3, 128);
                if (tid == 0) {
                    tc_wait(yread, c & 1, gone, a.ctl);   // Y makes room for dM
                    tc_fence_after();
                    issue_ts<3, NT, 2, DC>(tm + fwd_tmem::D, tm + fwd_tmem::SP, 32, stage, L::HALVES * kq_half, kq_half,
                                           mma_desc(128, DK, false, true), mn_major);
                    mma_commit(bs);
                    if (!kEarly && c > 0) tc_wait(oread, (c - 1) & 1, gone, a.ctl);
                    tc_fence_after();
                    issue_ts<L::PT, L::PT, L::PT - 1, DC>(tm + fwd_tmem::O, tm + u_at, 32, stage + L::P_AT, TILE, 16,
                                                          mma_desc(128, 64), tile_k);
                    mma_commit(bo);
                    mma_commit(empty + st);
                }
                __syncwarp();
            } else {
                if (c > 0) write_o(c - 1);
                tc_wait_warp(by, c & 1, gone, a.ctl);
                uint32_t r[DC];
                tmem_ld32(tm + fwd_tmem::D + lane_base, r);
                tmem_ld32(tm + fwd_tmem::D + lane_base + 32, r + 32);
                tmem_wait_ld();
#pragma unroll
                for (int t = 0; t < DC; ++t) y[t] = a.scale * gt.grown[t] * __uint_as_float(r[t]);
                tc_fence_before();
                mbar_arrive(yread);
            }
        }
        if (chunks > 0) {
            advance(chunks - 1);
            if (wg == 1) write_o(chunks - 1);
        }
        if (a.fin && in)
#pragma unroll
            for (int i = 0; i < HALF; ++i)
                if (col0 + i < a.Dk) a.fin[state + (size_t)(col0 + i) * a.Dv + dv] = m[i];
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free_all(tm);
}

}  // namespace qs
