// delta_fwd_tc.cuh -- forward of the gated delta rule on the tensor cores.
//
// One CTA walks the chunks of one (sequence, value head).  Everything that the
// chain of states goes through is laid out transposed: the state M^T [dv][dk], the
// errors e^T [dv][t] and so on have one value row dv per tensor-memory lane, so
// one thread owns one row of every product of the chain, and no value crosses
// threads between two of them.  Three warpgroups:
//
//   prep    one chunk ahead: loads K, Q and V, the decays, Gram products [K;Q] K^T,
//           T = (1 + A diag(beta))^-1 (32 x 32 blocks by substitution, the corner as
//           -T22 A21 T11), and writes T and P as operands;
//   chain   X = M^T K^T;  e = (v - exp(G) X) T^T;  M' = exp(G_C) M + (beta left e)^T K
//   out     Y = M^T Q^T;  o = exp(G) Y + U P^T; and half of the state's conversion
//
// The state stays in tensor memory in fp32, where its update accumulates.
//
// Bound: instruction issue and the chain's latency.  Per chunk of 64 steps the
// chain is three products after each other (D = 128: 2.1 + 1 + 2.1 MFLOP, in 3 to 6
// passes) with conversions to terms between them.  Loops over 32 columns rather
// than 64 unrolled ones keep the three roles' code in the instruction cache.
#pragma once

#include <type_traits>

#include "delta_common.cuh"
#include "tensor_core.cuh"

namespace qs {

// Gates of one chunk in shared memory.
struct __align__(16) ChunkGates {
    Sum2 sum[DC];                          // G_t
    float beta[DC], grown[DC], left[DC];   // beta_t, exp(G_t), exp(G_C - G_t)
    float mid[DC / 2];                     // exp(G_31 - G_s), s < 32
    float whole;                           // exp(G_C)
};

// A lane's two steps of a chunk's gates as they are read (one warp per chunk).
struct RawGates {
    float g[2], beta[2];
};
__device__ __forceinline__ RawGates read_gates(const DeltaArgs &a, const Seq &seq, long long t0, int head) {
    const int lane = threadIdx.x % 32;
    RawGates r;
    const long long left = seq.len - t0, row = (seq.b * a.S + seq.s0 + t0) * a.Hv + head;
    const int i0 = 2 * lane < left ? 2 * lane : 0, i1 = 2 * lane + 1 < left ? 2 * lane + 1 : 0;
    if (a.gate16) {
        const __nv_bfloat16 *g = static_cast<const __nv_bfloat16 *>(a.g) + row, *be = static_cast<const __nv_bfloat16 *>(a.beta) + row;
        const __nv_bfloat16 x = g[(long long)i0 * a.Hv], y = g[(long long)i1 * a.Hv], z = be[(long long)i0 * a.Hv], w = be[(long long)i1 * a.Hv];
        r = {{__bfloat162float(x), __bfloat162float(y)}, {__bfloat162float(z), __bfloat162float(w)}};
    } else {
        const float *g = static_cast<const float *>(a.g) + row, *be = static_cast<const float *>(a.beta) + row;
        r = {{g[(long long)i0 * a.Hv], g[(long long)i1 * a.Hv]}, {be[(long long)i0 * a.Hv], be[(long long)i1 * a.Hv]}};
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (2 * lane + i >= left) r.g[i] = r.beta[i] = 0.f;
    return r;
}

// One warp fills the gates of a chunk.
__device__ __forceinline__ void warp_gates(ChunkGates &s, const RawGates &raw) {
    const int lane = threadIdx.x % 32;
    Sum2 s0, s1;
    chunk_sums(clamp_gate(raw.g[0]), clamp_gate(raw.g[1]), &s0, &s1);
    const Sum2 end = {__shfl_sync(0xffffffffu, s1.hi, 31), __shfl_sync(0xffffffffu, s1.lo, 31)};
    const Sum2 mid = {__shfl_sync(0xffffffffu, s1.hi, 15), __shfl_sync(0xffffffffu, s1.lo, 15)};
    const int t = 2 * lane;
    s.sum[t] = s0, s.sum[t + 1] = s1;
    s.beta[t] = raw.beta[0], s.beta[t + 1] = raw.beta[1];
    s.grown[t] = decay(s0, {0.f, 0.f}), s.grown[t + 1] = decay(s1, {0.f, 0.f});
    s.left[t] = decay(end, s0), s.left[t + 1] = decay(end, s1);
    if (lane < 16) s.mid[t] = decay(mid, s0), s.mid[t + 1] = decay(mid, s1);
    if (lane == 31) s.whole = s.grown[63];
}

// Shared memory of the walks.  A tile is 64 rows x 64 values of bfloat16 (8 KB).
// K and Q of a stage: [term][half of D]{K tile, Q tile}; then a third tensor's rows
// [64][128] as they are (V; d_o in the backward), T and P.
constexpr uint32_t TILE = 8192;
constexpr int FLD = 68;   // padded rows of a 64 x 64 fp32 matrix (16-byte aligned)

template <typename T, int NT, int DK, int STAGES>
struct WalkLayout {
    static constexpr int HALVES = DK / 64;
    static constexpr uint32_t KQ = NT * HALVES * 2 * TILE;   // bytes of K and Q
    static constexpr int PT = NT == 1 ? 2 : 3;               // terms of P and U (o's precision)
    static constexpr uint32_t V_AT = KQ, T_AT = V_AT + DC * 128 * sizeof(T), P_AT = T_AT + 3 * TILE, STAGE = P_AT + PT * TILE;
    static constexpr uint32_t F_AT = STAGES * STAGE, Y_AT = F_AT + DC * FLD * 4;
    static constexpr uint32_t GATES_AT = Y_AT + 32 * 36 * 4;
    static constexpr uint32_t BARS_AT = GATES_AT + STAGES * sizeof(ChunkGates);
    static constexpr uint32_t BYTES = BARS_AT + 256 + 1024;   // + alignment of the tiles to 1024 bytes
    static_assert(BYTES <= 232448, "227 KB of shared memory");
    static_assert(BYTES > 116736, "one CTA per SM: it takes all of the tensor memory");
};

// Rows of one head into tiles as bfloat16 terms, `half` bytes from one half of D to
// the next and `term` from one term; zeros past the sequence and past D.  bfloat16
// rows are copied asynchronously.
template <typename T, int NT, int DK>
__device__ __forceinline__ void load_rows(uint32_t tiles, uint32_t half, uint32_t term, const void *p, const qsh::Strides &st,
                                          const Seq &seq, long long t0, int head, int D, int tid) {
    constexpr int UNITS = DK / 8, STEP = 128 / UNITS;   // 16-byte units of bfloat16 in a row; rows per round
    const int u = tid % UNITS, r0 = tid / UNITS;
    const T *base = static_cast<const T *>(p) + seq.b * st.b + (seq.s0 + t0) * st.s + (long long)head * st.h;
    const long long left = seq.len - t0;
    const uint32_t at0 = tiles + (uint32_t)(u / 8) * half;
#pragma unroll 4
    for (int r = r0; r < DC; r += STEP) {
        const bool in = r < left && u * 8 < D;
        const T *src = base + (in ? r * st.s + u * 8 : 0);
        const uint32_t at = at0 + swizzled(r, u % 8);
        if constexpr (NT == 1) {
            cp_async16_or_zero(at, src, in);
        } else {
            float4 x = q_zero(), y = q_zero();
            if (in) x = load4(src), y = load4(src + 4);
            uint32_t t[4][3];
            split2<3>(x.x, x.y, t[0]), split2<3>(x.z, x.w, t[1]), split2<3>(y.x, y.y, t[2]), split2<3>(y.z, y.w, t[3]);
#pragma unroll
            for (int j = 0; j < 3; ++j)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + j * term), "r"(t[0][j]), "r"(t[1][j]),
                             "r"(t[2][j]), "r"(t[3][j])
                             : "memory");
        }
    }
}

// Rows of one head as they are, [64][128], zeros past the sequence and past D.
template <typename T>
__device__ __forceinline__ void load_plain(uint32_t dst, const void *p, const qsh::Strides &st, const Seq &seq, long long t0, int head,
                                           int D, int tid) {
    constexpr int PER = 16 / sizeof(T), UNITS = 128 / PER, STEP = 128 / UNITS;
    const int u = tid % UNITS, r0 = tid / UNITS;
    const T *base = static_cast<const T *>(p) + seq.b * st.b + (seq.s0 + t0) * st.s + (long long)head * st.h;
    const long long left = seq.len - t0;
#pragma unroll 4
    for (int r = r0; r < DC; r += STEP) {
        const bool in = r < left && u * PER < D;
        cp_async16_or_zero(dst + r * 128 * sizeof(T) + u * 16, base + (in ? r * st.s + u * PER : 0), in);
    }
}

// Brings a chunk's rows of one head into L2 ahead of their use.
template <typename T>
__device__ __forceinline__ void prefetch_rows(const void *p, const qsh::Strides &st, const Seq &seq, long long t0, int head, int D,
                                              int tid) {
    constexpr int LINE = 128 / sizeof(T);
    const int r = tid % DC;
    if (t0 + r < seq.len)
        for (int x = tid / DC * LINE; x < D; x += 2 * LINE)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T *>(p) + seq.b * st.b + (seq.s0 + t0 + r) * st.s +
                                                          (long long)head * st.h + x));
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

// tf [64][FLD], strictly lower triangular (zeros on and above the diagonal inside
// its diagonal blocks), becomes (1 + tf)^-1 on and below the diagonal blocks; 128
// threads (barrier `bar`).  yf: 32 x 36 of scratch.
__device__ __forceinline__ void invert_64(float *tf, float *yf, int tid, int bar) {
    const int blk = tid / 32, j = tid % 32;
    if (blk < 2) {   // a diagonal block per warp, a column per thread, by substitution
        float *a = tf + blk * 32 * (FLD + 1);
        float2 x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            float2 s = make_float2(0.f, 0.f), s1 = make_float2(0.f, 0.f);
#pragma unroll
            for (int m = 0; m < i; m += 4) {   // terms past i meet zeros
                const float4 r = *reinterpret_cast<const float4 *>(a + i * FLD + m);
                s = fma2(make_float2(r.x, r.y), x[m / 2], s);
                if (m + 2 < i) s1 = fma2(make_float2(r.z, r.w), x[m / 2 + 1], s1);
            }
            const float v = (i == j ? 1.f : 0.f) - ((s.x + s1.x) + (s.y + s1.y));
            if (i % 2) x[i / 2].y = v;
            else x[i / 2].x = v;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) a[i * FLD + j] = i % 2 ? x[i / 2].y : x[i / 2].x;
    }
    named_bar_sync(bar, 128);
    const int r = tid / 8 * 2, c = tid % 8 * 4;   // a 2 x 4 piece of the corner per thread
    auto corner = [&](const float *a, const float *b, int ldb, int last, float4 *out) {
        float2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int m = 0; m < last; m += 4) {
            const float4 p = *reinterpret_cast<const float4 *>(a + r * FLD + m);
            const float4 q = *reinterpret_cast<const float4 *>(a + (r + 1) * FLD + m);
            const float pp[4] = {p.x, p.y, p.z, p.w}, qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 v = *reinterpret_cast<const float4 *>(b + (m + k) * ldb + c);
                y[0] = fma2(make_float2(pp[k], pp[k]), make_float2(v.x, v.y), y[0]);
                y[1] = fma2(make_float2(pp[k], pp[k]), make_float2(v.z, v.w), y[1]);
                y[2] = fma2(make_float2(qq[k], qq[k]), make_float2(v.x, v.y), y[2]);
                y[3] = fma2(make_float2(qq[k], qq[k]), make_float2(v.z, v.w), y[3]);
            }
        }
        out[0] = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
        out[1] = make_float4(y[2].x, y[2].y, y[3].x, y[3].y);
    };
    float4 y[2];
    corner(tf + 32 * FLD, tf, FLD, 32, y);   // A21 T11 (T11 holds zeros above its diagonal)
    store4(yf + r * 36 + c, y[0]);
    store4(yf + (r + 1) * 36 + c, y[1]);
    named_bar_sync(bar, 128);
    corner(tf + 32 * FLD + 32, yf, 36, (tid / 32 + 1) * 8, y);   // T22 is lower triangular
    store4(tf + (32 + r) * FLD + c, make_float4(-y[0].x, -y[0].y, -y[0].z, -y[0].w));
    store4(tf + (33 + r) * FLD + c, make_float4(-y[1].x, -y[1].y, -y[1].z, -y[1].w));
    named_bar_sync(bar, 128);
}

// Writes the rows of tf as the terms of T (what lies above the diagonal blocks stays).
__device__ __forceinline__ void store_inverse(uint32_t tiles, const float *tf, int tid) {
    const int r = tid / 2;   // two 16-byte units of an upper row, four of a lower one, per thread
#pragma unroll 1
    for (int u = (tid & 1) * (r < 32 ? 2 : 4), e = u + (r < 32 ? 2 : 4); u < e; ++u) {
        float x[8];
        const float4 p = *reinterpret_cast<const float4 *>(tf + r * FLD + u * 8);
        const float4 q = *reinterpret_cast<const float4 *>(tf + r * FLD + u * 8 + 4);
        x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w, x[4] = q.x, x[5] = q.y, x[6] = q.z, x[7] = q.w;
        store_terms<3>(tiles, r, u, x);
    }
}

// The Gram product [K;Q] K^T of a stage into tensor memory; one thread.
template <int NT, int DK>
__device__ __forceinline__ void issue_gram(uint32_t d, uint32_t stage) {
    constexpr uint32_t id = mma_desc(128, 64);
    const uint64_t base = smem_desc(stage, 16, 1024);   // its address field takes offsets without a carry
    bool add = false;
#pragma unroll
    for (int i = NT - 1; i >= 0; --i)
#pragma unroll
        for (int j = NT - 1; j >= 0; --j) {
            if (i + j > 2) continue;
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
                const uint32_t at = (k / 4) * 2 * TILE + (k % 4) * 32;
                mma_ss(d, base + ((i * (DK / 64) * 2 * TILE + at) >> 4), base + ((j * (DK / 64) * 2 * TILE + at) >> 4), id, add);
                add = true;
            }
        }
}

// One row of the Gram product (thread tid: row tid % 64 of K K^T, or of Q K^T from
// 64 on) times the decays: f(column, 16 values) for the 16-column pieces that hold
// any of s <= t; values past the diagonal are zero.  Below the warp's diagonal
// block D_ts = exp(G_t - G_31) exp(G_31 - G_s), both at most one: no exp per value.
template <typename F>
__device__ __forceinline__ void gram_rows(uint32_t g_at, const ChunkGates &gt, int tid, const F &f) {
    const int t = tid % 64, wb = t / 32;
    const Sum2 mine = gt.sum[t];
    const float row = wb ? decay(mine, gt.sum[31]) : 0.f;
#pragma unroll 1
    for (int h = 0; h <= wb; ++h)
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
            const int s0 = h * 32 + p * 16;
            uint32_t g[16];
            float x[16];
            __syncwarp();
            tmem_ld16(g_at + s0, g);
            tmem_wait_ld();
            if (h < wb) {
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 m = *reinterpret_cast<const float4 *>(&gt.mid[s0 + i]);
                    x[i] = __uint_as_float(g[i]) * (m.x * row), x[i + 1] = __uint_as_float(g[i + 1]) * (m.y * row);
                    x[i + 2] = __uint_as_float(g[i + 2]) * (m.z * row), x[i + 3] = __uint_as_float(g[i + 3]) * (m.w * row);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const Sum2 o = gt.sum[s0 + i];
                    const float d = (mine.hi - o.hi) + (mine.lo - o.lo);
                    x[i] = s0 + i <= t ? __uint_as_float(g[i]) * exp2_fast(s0 + i <= t ? d : 0.f) : 0.f;
                }
            }
            f(s0, x);
        }
}

// Issues D[128 x N] (+)= sum over term pairs of A[tmem] B[smem], K values of K;
// one thread.  `a_at(i, k)` gives the column of K step k of A's term i, `b_at(k)` the
// byte offset of B's; B's terms are `b_term` bytes apart.  Pairs i + j <= LAST.
template <int TA, int TB, int LAST, int K, typename A, typename Bo>
__device__ __forceinline__ void issue_ts(uint32_t d, const A &a_at, uint32_t b, uint32_t b_term, uint32_t lbo, uint32_t idesc,
                                         const Bo &b_at, bool add = false) {
    const uint64_t base = smem_desc(b, lbo, 1024);
#pragma unroll
    for (int i = TA - 1; i >= 0; --i)   // small terms first
#pragma unroll
        for (int j = TB - 1; j >= 0; --j) {
            if (i + j > LAST) continue;
#pragma unroll
            for (int k = 0; k < K / 16; ++k) {
                mma_ts(d, a_at(i, k), base + ((j * b_term + b_at(k)) >> 4), idesc, add);
                add = true;
            }
        }
}

// Tensor-memory columns of the forward walk.  With bfloat16 inputs (two terms
// for o) the operands are placed so that Y and U P^T run while the chain converts:
// the terms of v - exp(G) X take the place of M's third term, which only X needs,
// and U that of e.  With fp32 inputs Y needs all of M's terms, and the chain waits.
namespace fwd_tmem {
constexpr uint32_t M = 0;      // the state (128)
constexpr uint32_t SP = 128;   // terms of M (3 x 64), later of beta left e (3 x 32)
constexpr uint32_t X = 320;    // X, then e, then (bfloat16) U
constexpr uint32_t O = 384;    // Y, then o
constexpr uint32_t G = 448;    // Gram products
}  // namespace fwd_tmem

constexpr int kWalkThreads = 384;

// Barriers and flags of a walk's CTA.
struct WalkBars {
    uint64_t full[2], empty[2], x, y, e, s, o, g, yread, oread;
    uint32_t tmem;
    int gone;
};

template <typename T, int NT, int DK, int STAGES>
__global__ void __launch_bounds__(kWalkThreads, 1) delta_fwd_tc_kernel(const __grid_constant__ DeltaArgs a) {
    using L = WalkLayout<T, NT, DK, STAGES>;
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
            mbar_init(&bar.empty[i], 1);
        }
        for (uint64_t *b : {&bar.x, &bar.y, &bar.e, &bar.s, &bar.o, &bar.g}) mbar_init(b, 1);
        mbar_init(&bar.yread, 128);
        mbar_init(&bar.oread, 128);
        *gone = 0;
        fence_mbar_init();
    }
    // T and P are zero above the diagonal blocks, where prep never writes.
    for (int st = 0; st < STAGES; ++st)
        for (uint32_t i = threadIdx.x; i < (3 + L::PT) * TILE / 16; i += kWalkThreads) {
            const uint32_t z[4] = {0, 0, 0, 0};
            st_shared16(sm32 + st * L::STAGE + L::T_AT + i * 16, z);
        }
    if (warp == 0) tmem_alloc_all(&bar.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = bar.tmem;
    const uint32_t tl = tm + ((uint32_t)(warp % 4 * 32) << 16);   // this warp's lanes

    if (wg == 2) {
        // ------------------------------------------------------------ prep
        float *tf = reinterpret_cast<float *>(sm + L::F_AT);
        float *yf = reinterpret_cast<float *>(sm + L::Y_AT);
        RawGates raw_gates = {};
        if (tid < 32 && chunks > 0) raw_gates = read_gates(a, seq, 0, head);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int st = c % STAGES;
            const uint32_t stage = sm32 + st * L::STAGE;
            const long long t0 = (long long)c * DC;
            ChunkGates &gt = gates[st];
            tc_wait_warp(&bar.empty[st], ((c / STAGES) & 1) ^ 1, gone, a.ctl);
            load_rows<T, NT, DK>(stage, 2 * TILE, L::HALVES * 2 * TILE, a.k, a.sk, seq, t0, kh, a.Dk, tid);
            load_rows<T, NT, DK>(stage + TILE, 2 * TILE, L::HALVES * 2 * TILE, a.q, a.sq, seq, t0, kh, a.Dk, tid);
            load_plain<T>(stage + L::V_AT, a.v, a.sv, seq, t0, head, a.Dv, tid);
            if (c + 1 < chunks) {
                prefetch_rows<T>(a.k, a.sk, seq, t0 + DC, kh, a.Dk, tid);
                prefetch_rows<T>(a.q, a.sq, seq, t0 + DC, kh, a.Dk, tid);
                prefetch_rows<T>(a.v, a.sv, seq, t0 + DC, head, a.Dv, tid);
            }
            if (tid < 32) {
                warp_gates(gt, raw_gates);
                if (c + 1 < chunks) raw_gates = read_gates(a, seq, t0 + DC, head);
            }
            cp_async_wait_all();
            fence_proxy_async_smem();
            named_bar_sync(2, 128);
            if (tid == 0) {
                tc_fence_after();
                issue_gram<NT, DK>(tm + fwd_tmem::G, stage);
                mma_commit(&bar.g);
            }
            __syncwarp();
            tc_wait_warp(&bar.g, c & 1, gone, a.ctl);
            gram_rows(tl + fwd_tmem::G, gt, tid, [&](int s0, float *x) {
                const int t = tid % 64;
                if (tid < 64) {   // A_ts beta_s, zero on the diagonal
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 be = *reinterpret_cast<const float4 *>(&gt.beta[s0 + i]);
                        const float b4[4] = {be.x, be.y, be.z, be.w};
                        float y[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) y[j] = s0 + i + j == t ? 0.f : x[i + j] * b4[j];
                        store4(tf + t * FLD + s0 + i, make_float4(y[0], y[1], y[2], y[3]));
                    }
                } else {          // P_ts
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] *= a.scale;
                    store_terms<L::PT>(stage + L::P_AT, t, s0 / 8, x);
                    store_terms<L::PT>(stage + L::P_AT, t, s0 / 8 + 1, x + 8);
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
        constexpr int HALF = DK / 2;             // columns of the state per thread
        constexpr bool kEarly = NT == 1;
        constexpr uint32_t kq_half = 2 * TILE, kq_term = L::HALVES * kq_half;
        const int dv = tid, col0 = wg * HALF;
        const bool in = dv < a.Dv;
        const size_t state = ((size_t)n * a.Hv + head) * a.Dk * a.Dv + dv;
        auto k_major = [](int k) { return (uint32_t)((k / 4) * 2 * TILE + (k % 4) * 32); };   // K or Q [t][dk]: K steps along dk
        auto mn_major = [](int k) { return (uint32_t)(k * 2048); };                          // K [t][dk]: K steps along t
        auto tile_k = [](int k) { return (uint32_t)(k * 32); };                              // T or P
        auto m_terms = [&](int i, int k) { return tm + fwd_tmem::SP + i * 64 + k * 8; };
        // Terms of v - exp(G) X: over M's third term and O, or over M's terms once Y is done.
        auto e0_at = [](int j) { return !kEarly ? fwd_tmem::SP + j * 32 : j < 2 ? fwd_tmem::SP + 128 + j * 32 : fwd_tmem::O; };
        // U: where e stood, each 32 columns of e giving way to its own terms, or beyond beta left e's.
        auto u_at = [](int j, int t) { return kEarly ? fwd_tmem::X + t / 32 * 32 + j * 16 + t % 32 / 2 : fwd_tmem::SP + 96 + j * 32 + t / 2; };
        const long long row0 = seq.b * a.S + seq.s0;

#pragma unroll 1
        for (int h = 0; h < HALF; h += 16) {
            uint32_t r[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                r[i] = __float_as_uint(a.init && in && col0 + h + i < a.Dk ? __ldg(a.init + state + (size_t)(col0 + h + i) * a.Dv) : 0.f);
            __syncwarp();
            tmem_st16(tl + fwd_tmem::M + col0 + h, r);
        }
        tmem_wait_st();

        // o of chunk c.
        auto write_o = [&](int c) {
            tc_wait_warp(&bar.o, c & 1, gone, a.ctl);
            const int left = (int)min((long long)DC, seq.len - (long long)c * DC);
            T *out = static_cast<T *>(a.o) + ((size_t)(row0 + (long long)c * DC) * a.Hv + head) * a.Dv + dv;
            const size_t step = (size_t)a.Hv * a.Dv;
#pragma unroll 1
            for (int h = 0; h < DC; h += 32) {
                uint32_t r[32];
                tmem_ld32(tl + fwd_tmem::O + h, r);
                tmem_wait_ld();
                if (h == 32) {
                    tc_fence_before();
                    mbar_arrive(&bar.oread);
                }
                if (in)
#pragma unroll
                    for (int i = 0; i < 32; ++i, out += step)
                        if (h + i < left) store1(out, __uint_as_float(r[i]));
                __syncwarp();
            }
        };

#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const int st = c % STAGES;
            const uint32_t stage = sm32 + st * L::STAGE;
            const ChunkGates &gt = gates[st];
            const int left = (int)min((long long)DC, seq.len - (long long)c * DC);
            tc_wait_warp(&bar.full[st], (c / STAGES) & 1, gone, a.ctl);
            if (c > 0) tc_wait_warp(&bar.s, (c - 1) & 1, gone, a.ctl);
            if (!kEarly && c > 0) tc_wait_warp(&bar.o, (c - 1) & 1, gone, a.ctl);   // U lies where M's terms go
            float *carry = a.carries ? a.carries + ((size_t)(seq.slot0 + c) * a.Hv + head) * a.Dk * a.Dv + dv : nullptr;
#pragma unroll 1
            for (int h = 0; h < HALF; h += 32) {   // the state: terms, and scaled for its update
                uint32_t r[32], t[3][16];
                tmem_ld32(tl + fwd_tmem::M + col0 + h, r);
                tmem_wait_ld();
                const float2 w = make_float2(gt.whole, gt.whole);
                if (carry && in) {
                    float *out = carry + (size_t)(col0 + h) * a.Dv;
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
                for (int j = 0; j < 3; ++j) tmem_st16(tl + fwd_tmem::SP + j * 64 + (col0 + h) / 2, t[j]);
                tmem_st32(tl + fwd_tmem::M + col0 + h, r);
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, 256);
            auto issue_y = [&] {
                issue_ts<L::PT, NT, L::PT - 1, DK>(tm + fwd_tmem::O, m_terms, stage + TILE, kq_term, 16, mma_desc(128, 64), k_major);
                mma_commit(&bar.y);
            };
            if (wg == 0) {
                if (tid == 0) {
                    tc_fence_after();
                    issue_ts<3, NT, 2, DK>(tm + fwd_tmem::X, m_terms, stage, kq_term, 16, mma_desc(128, 64), k_major);
                    mma_commit(&bar.x);
                    if (!kEarly) {
                        if (c > 0) tc_wait(&bar.oread, (c - 1) & 1, gone, a.ctl);
                        tc_fence_after();
                        issue_y();
                    }
                }
                __syncwarp();
                tc_wait_warp(&bar.x, c & 1, gone, a.ctl);
                if (kEarly && c > 0) tc_wait_warp(&bar.oread, (c - 1) & 1, gone, a.ctl);
                if (!kEarly) tc_wait_warp(&bar.y, c & 1, gone, a.ctl);
                const T *vs = reinterpret_cast<const T *>(sm + st * L::STAGE + L::V_AT) + dv;
#pragma unroll 1
                for (int h = 0; h < DC; h += 32) {
                    uint32_t r[32], t[3][16];
                    tmem_ld32(tl + fwd_tmem::X + h, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 g = *reinterpret_cast<const float2 *>(&gt.grown[h + 2 * i]);
                        const float2 v = make_float2(to_float(vs[(h + 2 * i) * 128]), to_float(vs[(h + 2 * i + 1) * 128]));
                        uint32_t p[3];
                        split2<3>(fma2(make_float2(-__uint_as_float(r[2 * i]), -__uint_as_float(r[2 * i + 1])), g, v), p);
                        t[0][i] = p[0], t[1][i] = p[1], t[2][i] = p[2];
                    }
#pragma unroll
                    for (int j = 0; j < 3; ++j) tmem_st16(tl + e0_at(j) + h / 2, t[j]);
                }
                tmem_wait_st();
                tc_fence_before();
                named_bar_sync(3, 128);
                if (tid == 0) {
                    tc_fence_after();
                    issue_ts<3, 3, 2, DC>(tm + fwd_tmem::X, [&](int i, int k) { return tm + e0_at(i) + k * 8; }, stage + L::T_AT, TILE, 16,
                                          mma_desc(128, 64), tile_k);
                    mma_commit(&bar.e);
                    if (kEarly) issue_y();   // (in order after e, whose operand lies in O)
                }
                __syncwarp();
                tc_wait_warp(&bar.e, c & 1, gone, a.ctl);
                float *eo = a.errors ? a.errors + ((size_t)(row0 + (long long)c * DC) * a.Hv + head) * a.Dv + dv : nullptr;
                const size_t step = (size_t)a.Hv * a.Dv;
#pragma unroll 1
                for (int h = 0; h < DC; h += 32) {
                    uint32_t r[32], t[3][16];
                    tmem_ld32(tl + fwd_tmem::X + h, r);
                    tmem_wait_ld();
                    if (eo && in) {
                        float *out = eo + h * step;
#pragma unroll
                        for (int i = 0; i < 32; ++i, out += step)
                            if (h + i < left) *out = __uint_as_float(r[i]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 be = *reinterpret_cast<const float2 *>(&gt.beta[h + 2 * i]);
                        const float2 u = mul2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), be);
                        r[2 * i] = __float_as_uint(u.x), r[2 * i + 1] = __float_as_uint(u.y);
                        uint32_t p[3];
                        split2<L::PT>(u, p);
#pragma unroll
                        for (int j = 0; j < L::PT; ++j) t[j][i] = p[j];
                    }
#pragma unroll
                    for (int j = 0; j < L::PT; ++j) tmem_st16(tl + u_at(j, h), t[j]);
                    if (kEarly && h == 0) tc_wait_warp(&bar.y, c & 1, gone, a.ctl);   // Y reads M's first terms
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 lf = *reinterpret_cast<const float2 *>(&gt.left[h + 2 * i]);
                        uint32_t p[3];
                        split2<3>(mul2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), lf), p);
                        t[0][i] = p[0], t[1][i] = p[1], t[2][i] = p[2];
                    }
#pragma unroll
                    for (int j = 0; j < 3; ++j) tmem_st16(tl + fwd_tmem::SP + j * 32 + h / 2, t[j]);
                }
                tmem_wait_st();
                tc_fence_before();
                named_bar_sync(3, 128);
                if (tid == 0) {
                    tc_fence_after();
                    issue_ts<3, NT, 2, DC>(tm + fwd_tmem::M, [&](int i, int k) { return tm + fwd_tmem::SP + i * 32 + k * 8; }, stage, kq_term,
                                           kq_half, mma_desc(128, DK, false, true), mn_major, true);
                    mma_commit(&bar.s);
                    tc_wait(&bar.yread, c & 1, gone, a.ctl);   // Y has been scaled
                    tc_fence_after();
                    issue_ts<L::PT, L::PT, L::PT - 1, DC>(tm + fwd_tmem::O, [&](int i, int k) { return tm + u_at(i, k * 16); },
                                                          stage + L::P_AT, TILE, 16, mma_desc(128, 64), tile_k, true);
                    mma_commit(&bar.o);
                    mma_commit(&bar.empty[st]);
                }
                __syncwarp();
            } else {
                if (c > 0) write_o(c - 1);
                tc_wait_warp(&bar.y, c & 1, gone, a.ctl);
#pragma unroll 1
                for (int h = 0; h < DC; h += 32) {   // scale exp(G) Y, on which U P^T adds up
                    uint32_t r[32];
                    tmem_ld32(tl + fwd_tmem::O + h, r);
                    tmem_wait_ld();
                    const float2 sc = make_float2(a.scale, a.scale);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 g = mul2(*reinterpret_cast<const float2 *>(&gt.grown[h + 2 * i]), sc);
                        const float2 y = mul2(make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), g);
                        r[2 * i] = __float_as_uint(y.x), r[2 * i + 1] = __float_as_uint(y.y);
                    }
                    tmem_st32(tl + fwd_tmem::O + h, r);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bar.yread);
            }
        }
        if (chunks > 0) {
            tc_wait_warp(&bar.s, (chunks - 1) & 1, gone, a.ctl);
            if (wg == 1) write_o(chunks - 1);
        }
        if (a.fin)
#pragma unroll 1
            for (int h = 0; h < HALF; h += 16) {
                uint32_t r[16];
                __syncwarp();
                tmem_ld16(tl + fwd_tmem::M + col0 + h, r);
                tmem_wait_ld();
                if (in)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (col0 + h + i < a.Dk) a.fin[state + (size_t)(col0 + h + i) * a.Dv] = __uint_as_float(r[i]);
            }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_free_all(tm);
}

}  // namespace qs
