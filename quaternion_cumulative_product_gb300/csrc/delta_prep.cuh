// delta_prep.cuh -- what the two walks of the delta rule (the forward over chunks,
// the backward's chain of cotangents) share: the gates and operands of a chunk,
// prepared one chunk ahead by two warpgroups.
//
// Per chunk: K, Q and a third tensor (V, or dO in the backward) as tiles, the
// decays, the Gram products [K;Q] K^T, P, and T = (1 + N)^-1 for N = A diag(beta)
// (forward) or diag(beta) A (backward): 16 x 16 diagonal blocks by substitution, then
// twice the corner of a block as -T22 N21 T11.  All in fp32; T and P leave as terms.
//
// bfloat16 tensors come by TMA (swizzled boxes of 64 steps x 64 values) into a ring of
// chunks that the walk refills: three for D <= 64, where a chunk's Gram products run while
// the chunk before is inverted (139 instead of 152 us for a segment walk of 1 x 16384 x 16
// x 64), two for D = 128 (three leave room for a single T: 390 instead of 356 us at 8 x
// 4096 x 16 x 128).  fp32 tensors go through registers, which split them, one chunk at a time:
// their terms take three times the space.
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

// RULE, here and in the kernels: the gated delta rule; else linear attention with a decay,
// which is the rule without its errors (e = v, no T) and without beta (1).

// A lane's two steps of a chunk's gates as they are read (one warp per chunk).
struct RawGates {
    float g[2], beta[2];
};
template <bool RULE = true>
__device__ __forceinline__ RawGates read_gates(const DeltaArgs &a, const Seq &seq, long long t0, int head) {
    const int lane = threadIdx.x % 32;
    RawGates r;
    const long long left = seq.len - t0, row = (seq.b * a.S + seq.s0 + t0) * a.Hv + head;
    const int i0 = 2 * lane < left ? 2 * lane : 0, i1 = 2 * lane + 1 < left ? 2 * lane + 1 : 0;
    if constexpr (!RULE) {
        r = {{load_any(a.g, a.gate16, row + (long long)i0 * a.Hv), load_any(a.g, a.gate16, row + (long long)i1 * a.Hv)}, {1.f, 1.f}};
    } else if (a.gate16) {
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

// A tile is 64 rows x 64 values of bfloat16 (8 KB, 128-byte swizzle).
constexpr uint32_t TILE = 8192;
constexpr int FLD = 68;   // padded rows of a 64 x 64 fp32 matrix (16-byte aligned)

__device__ __forceinline__ void st_shared16(uint32_t at, const uint32_t *v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// Rows of one head into tiles as bfloat16 terms, `half` bytes from one half of D to
// the next and `term` from one term; zeros past the sequence and past D.  bfloat16
// rows are copied asynchronously.  THREADS threads.
template <typename T, int NT, int DK, int THREADS>
__device__ __forceinline__ void load_rows(uint32_t tiles, uint32_t half, uint32_t term, const void *p, const qsh::Strides &st,
                                          const Seq &seq, long long t0, int head, int D, int tid) {
    constexpr int UNITS = DK / 8, STEP = THREADS / UNITS;   // 16-byte units of bfloat16 in a row; rows per round
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
            for (int j = 0; j < 3; ++j) {
                const uint32_t v[4] = {t[0][j], t[1][j], t[2][j], t[3][j]};
                st_shared16(at + j * term, v);
            }
        }
    }
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

constexpr int kPrepThreads = 256;

// tf [64][FLD], strictly lower triangular (zeros on and above the diagonal inside
// its 16 x 16 and 32 x 32 diagonal blocks), becomes (1 + tf)^-1 on and below the
// diagonal of its 32 x 32 blocks and in the lower corner (the upper one is scratch);
// kPrepThreads threads (barrier `bar`).
__device__ __forceinline__ void invert_64(float *tf, int tid, int bar) {
    float *yf = tf + 32;
    const int warp = tid / 32, j = tid % 32;
    if (warp < 4 && j < 16) {   // a diagonal block per half warp, a column per thread, by substitution
        float *a = tf + warp * 16 * (FLD + 1);
        float2 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
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
        __syncwarp(0xffffu);
#pragma unroll
        for (int i = 0; i < 16; ++i) a[i * FLD + j] = i % 2 ? x[i / 2].y : x[i / 2].x;
    }
    named_bar_sync(bar, kPrepThreads);
    {   // 16 -> 32: two corners, 1 x 2 values per thread
        const int b = tid / 128, r = tid % 128 / 8, c = tid % 8 * 2;
        float *d = tf + b * 32 * (FLD + 1), *y = yf + b * 16;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
            const float4 p = *reinterpret_cast<const float4 *>(d + (16 + r) * FLD + m);
            v = fma2(make_float2(p.x, p.x), *reinterpret_cast<const float2 *>(d + m * FLD + c), v);
            v = fma2(make_float2(p.y, p.y), *reinterpret_cast<const float2 *>(d + (m + 1) * FLD + c), v);
            v = fma2(make_float2(p.z, p.z), *reinterpret_cast<const float2 *>(d + (m + 2) * FLD + c), v);
            v = fma2(make_float2(p.w, p.w), *reinterpret_cast<const float2 *>(d + (m + 3) * FLD + c), v);
        }
        *reinterpret_cast<float2 *>(y + r * FLD + c) = v;
        named_bar_sync(bar, kPrepThreads);
        v = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < 16; m += 4) {
            const float4 p = *reinterpret_cast<const float4 *>(d + (16 + r) * FLD + 16 + m);
            v = fma2(make_float2(p.x, p.x), *reinterpret_cast<const float2 *>(y + m * FLD + c), v);
            v = fma2(make_float2(p.y, p.y), *reinterpret_cast<const float2 *>(y + (m + 1) * FLD + c), v);
            v = fma2(make_float2(p.z, p.z), *reinterpret_cast<const float2 *>(y + (m + 2) * FLD + c), v);
            v = fma2(make_float2(p.w, p.w), *reinterpret_cast<const float2 *>(y + (m + 3) * FLD + c), v);
        }
        *reinterpret_cast<float2 *>(d + (16 + r) * FLD + c) = make_float2(-v.x, -v.y);
    }
    named_bar_sync(bar, kPrepThreads);
    {   // 32 -> 64: 2 x 2 values per thread
        const int r = tid / 16 * 2, c = tid % 16 * 2;
        auto corner = [&](const float *a, const float *b, int ldb, float2 *v) {
            v[0] = v[1] = make_float2(0.f, 0.f);
#pragma unroll 2
            for (int m = 0; m < 32; m += 4) {
                const float4 p = *reinterpret_cast<const float4 *>(a + r * FLD + m);
                const float4 q = *reinterpret_cast<const float4 *>(a + (r + 1) * FLD + m);
                const float pp[4] = {p.x, p.y, p.z, p.w}, qq[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 w = *reinterpret_cast<const float2 *>(b + (m + k) * ldb + c);
                    v[0] = fma2(make_float2(pp[k], pp[k]), w, v[0]);
                    v[1] = fma2(make_float2(qq[k], qq[k]), w, v[1]);
                }
            }
        };
        float2 v[2];
        corner(tf + 32 * FLD, tf, FLD, v);
        *reinterpret_cast<float2 *>(yf + r * FLD + c) = v[0];
        *reinterpret_cast<float2 *>(yf + (r + 1) * FLD + c) = v[1];
        named_bar_sync(bar, kPrepThreads);
        corner(tf + 32 * FLD + 32, yf, FLD, v);
        *reinterpret_cast<float2 *>(tf + (32 + r) * FLD + c) = make_float2(-v[0].x, -v[0].y);
        *reinterpret_cast<float2 *>(tf + (33 + r) * FLD + c) = make_float2(-v[1].x, -v[1].y);
    }
    named_bar_sync(bar, kPrepThreads);
}

// Writes the rows of tf as the terms of T (what lies above the 32 x 32 diagonal blocks stays).
__device__ __forceinline__ void store_inverse(uint32_t tiles, const float *tf, int tid) {
#pragma unroll 1
    for (int i = tid; i < 32 * 4 + 32 * 8; i += kPrepThreads) {
        const int r = i < 128 ? i / 4 : 32 + (i - 128) / 8, u = i < 128 ? i % 4 : i % 8;
        float x[8];
        const float4 p = *reinterpret_cast<const float4 *>(tf + r * FLD + u * 8);
        const float4 q = *reinterpret_cast<const float4 *>(tf + r * FLD + u * 8 + 4);
        x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w, x[4] = q.x, x[5] = q.y, x[6] = q.z, x[7] = q.w;
        store_terms<3>(tiles, r, u, x);
    }
}

// Issues D (+)= sum over term pairs i + j <= LAST of A[smem] B[smem]; one thread.
// Terms are `a_term`, `b_term` bytes apart, `a_at(k)`, `b_at(k)` the offsets of K step k.
template <int TA, int TB, int LAST, int STEPS, typename Ao, typename Bo>
__device__ __forceinline__ void issue_ss(uint32_t d, uint64_t a, uint32_t a_term, uint64_t b, uint32_t b_term, uint32_t idesc,
                                         const Ao &a_at, const Bo &b_at, bool add = false) {
#pragma unroll 1
    for (int i = TA - 1; i >= 0; --i)   // small terms first
#pragma unroll 1
        for (int j = min(TB - 1, LAST - i); j >= 0; --j) {
            const uint64_t ai = a + ((i * a_term) >> 4), bj = b + ((j * b_term) >> 4);   // (address fields take offsets without a carry)
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                mma_ss(d, ai + (a_at(k) >> 4), bj + (b_at(k) >> 4), idesc, add);
                add = true;
            }
        }
}
// The same with A in tensor memory: terms `a_term` columns apart, K step k at a_at(k).  All
// pairs of terms, or all but the pair of first terms, or that one.
enum Pairs { kAllPairs, kSmallPairs, kFirstPair };
template <int TA, int TB, int LAST, int STEPS, typename Ao, typename Bo>
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a, uint32_t a_term, uint64_t b, uint32_t b_term, uint32_t idesc,
                                         const Ao &a_at, const Bo &b_at, bool add = false, Pairs pairs = kAllPairs) {
#pragma unroll 1
    for (int i = pairs == kFirstPair ? 0 : TA - 1; i >= 0; --i)
#pragma unroll 1
        for (int j = pairs == kFirstPair ? 0 : min(TB - 1, LAST - i); j >= (pairs == kSmallPairs && i == 0 ? 1 : 0); --j) {
            const uint64_t bj = b + ((j * b_term) >> 4);
            const uint32_t ai = a + i * a_term;
#pragma unroll
            for (int k = 0; k < STEPS; ++k) {
                mma_ts(d, ai + a_at(k), bj + (b_at(k) >> 4), idesc, add);
                add = true;
            }
        }
}

// Offsets of K step k (16 values of K).
struct KMajor {    // along the rows of [half][2 tiles of 64 rows]
    __device__ __forceinline__ uint32_t operator()(int k) const { return (uint32_t)((k / 4) * 2 * TILE + (k % 4) * 32); }
};
struct KMajor1 {   // along the rows of one tile
    __device__ __forceinline__ uint32_t operator()(int k) const { return (uint32_t)(k * 32); }
};
struct MNMajor {   // across the rows of a tile
    __device__ __forceinline__ uint32_t operator()(int k) const { return (uint32_t)(k * 2048); }
};
struct TmemK {     // 8 columns of a left operand in tensor memory
    __device__ __forceinline__ uint32_t operator()(int k) const { return (uint32_t)(k * 8); }
};

// Barriers and flags of a walk's CTA.
struct WalkBars {
    uint64_t full[2], empty[2], rows[3], x, e, s, o, g, drain[2];
    uint32_t tmem;
    int gone, fetched;   // chunks whose rows have been sent for
};

// Shared memory of a walk.  KS chunks of rows: K and Q [term][half of D]{K tile, Q tile},
// the third tensor [term][half of D]; S slots of T [3 terms] and P [PT terms].
template <int NT, int DK, int PT>
struct WalkLayout {
    static constexpr int KS = NT == 3 ? 1 : DK == 64 ? 3 : 2, S = NT == 3 ? 1 : 2;
    static constexpr int HALVES = DK / 64;
    static constexpr uint32_t KQ_TERM = HALVES * 2 * TILE, V_AT = NT * KQ_TERM, V_TERM = 2 * TILE, ROWS = V_AT + NT * V_TERM;
    static constexpr uint32_t T_AT = KS * ROWS, P_IN = 3 * TILE, SLOT = P_IN + PT * TILE;
    static constexpr uint32_t F_AT = T_AT + S * SLOT;
    static constexpr uint32_t GATES_AT = F_AT + DC * FLD * 4;
    static constexpr uint32_t BARS_AT = GATES_AT + 4 * sizeof(ChunkGates);
    static constexpr uint32_t NEED = BARS_AT + 256 + 1024;            // + alignment of the tiles to 1024 bytes
    static constexpr uint32_t BYTES = NEED > 117760 ? NEED : 117760;  // one CTA per SM: it takes all of the tensor memory
    static_assert(BYTES <= 232448, "227 KB of shared memory");
};

constexpr int kWalkThreads = 512;   // two warpgroups that walk, two of prep

// Which walk a CTA takes: sequence, head, segment.  SUM: the walk over a segment that
// sums it up as an affine map of the state (for all segments but the last; backward:
// but the first).  Its rows hold the segment's own part (from the zero state on) and, from
// row `map_from`, the map's columns (from the identity on, without inputs).
struct Walk {
    long long n;
    int head, seg, map_from;
    size_t at;   // (n * Hv + head) * segs + seg
    bool any;    // there is one (linear attention's cuts of packed sequences: the host knows a bound only)
};

// The sequence of CTA row i where packed sequences are walked longest first: the one that
// i others come before.  (All threads of the CTA call this.)
template <int THREADS>
__device__ __forceinline__ unsigned by_length(const int *offsets, long long N, long long S, unsigned i, int *chunks, int *before,
                                              volatile unsigned *mine) {   // (the last three: shared memory)
    const unsigned t = threadIdx.x % kMostOrdered, part = threadIdx.x / kMostOrdered;
    constexpr unsigned kParts = THREADS / kMostOrdered;
    if (part == 0) {
        chunks[t] = t < N ? (int)((seq_of(offsets, S, t).len + DC - 1) / DC) : -1;
        before[t] = 0;
    }
    __syncthreads();
    const int c = chunks[t];
    int n = 0;
#pragma unroll 8
    for (unsigned u = part; u < kMostOrdered; u += kParts) n += chunks[u] > c || (chunks[u] == c && u < t);
    atomicAdd(&before[t], n);   // (whole numbers: their order changes nothing)
    __syncthreads();
    if (part == 0 && before[t] == (int)i) *mine = t;
    __syncthreads();
    return *mine;
}

// The i-th segment of a packed batch whose long sequences are cut into segments of `most` chunks (the others,
// empty ones too, are one), false past the last: longest sequences first, or, of more than kMostOrdered sequences, at
// (first slot of the sequence) / most + n + segment.  All threads of the CTA.
template <int THREADS>
__device__ __forceinline__ bool cut_segment(const DeltaArgs &a, unsigned i, int *chunks, int *before, volatile unsigned *mine, Walk *w) {
    const int most = (int)a.seg_chunks;
    if (a.N > kMostOrdered) {
        long long lo = 0, hi = a.N;
        while (hi - lo > 1) {
            const long long mid = (lo + hi) / 2;
            if (seq_of(a, mid).slot0 / most + mid <= i) lo = mid;
            else hi = mid;
        }
        const Seq seq = seq_of(a, lo);
        const long long seg = (long long)i - (seq.slot0 / most + lo);
        w->n = lo, w->seg = (int)seg;
        return seg == 0 || (seg > 0 && is_cut(a, seq) && seg * most * DC < seq.len);
    }
    const unsigned t = threadIdx.x % kMostOrdered, part = threadIdx.x / kMostOrdered;
    constexpr unsigned kParts = THREADS / kMostOrdered;
    int *segs = chunks + kMostOrdered;
    if (part == 0) {
        chunks[t] = -1, segs[t] = 0;
        if (t < a.N) {
            const Seq seq = seq_of(a, t);
            chunks[t] = (int)((seq.len + DC - 1) / DC);
            segs[t] = is_cut(a, seq) ? (chunks[t] + most - 1) / most : 1;
        }
        before[t] = 0;
        if (t == 0) mine[0] = kMostOrdered;
    }
    __syncthreads();
    const int c = chunks[t];
    int n = 0;
#pragma unroll 8
    for (unsigned u = part; u < kMostOrdered; u += kParts) n += chunks[u] > c || (chunks[u] == c && u < t) ? segs[u] : 0;
    atomicAdd(&before[t], n);   // (whole numbers: their order changes nothing)
    __syncthreads();
    if (part == 0 && (int)i >= before[t] && (int)i < before[t] + segs[t]) mine[0] = t, mine[1] = i - before[t];
    __syncthreads();
    w->n = mine[0], w->seg = (int)mine[1];
    return mine[0] < kMostOrdered;
}

template <bool SUM, bool BWD, bool RULE = true>
__device__ __forceinline__ Walk walk_of(const DeltaArgs &a) {
    Walk w;
    unsigned i = blockIdx.x;
    w.map_from = 128;
    w.any = true;
    int segs = a.segs;
    if (SUM) {
        segs -= 1;
        if (a.Dk <= 64 && a.Dv <= 64) {
            w.map_from = 64;
        } else {   // own part and map in CTAs of their own
            if (i % 2) w.map_from = 0;
            i /= 2;
        }
    }
    w.head = i % a.Hv, i /= a.Hv;
    w.seg = i % segs + (SUM && BWD ? 1 : 0);
    w.n = i / segs;
    __shared__ int lengths[RULE ? 2 : 3][kMostOrdered];
    __shared__ unsigned mine[RULE ? 1 : 2];
    if (!RULE && a.uncut) w.any = cut_segment<kWalkThreads>(a, i, lengths[0], lengths[RULE ? 0 : 2], mine, &w);
    else if (!SUM && a.longest_first) w.n = by_length<kWalkThreads>(a.offsets, a.N, a.S, (unsigned)w.n, lengths[0], lengths[1], mine);
    w.at = ((size_t)w.n * a.Hv + w.head) * a.segs + w.seg;
    return w;
}

// The element (column x of dk) that this thread's row starts with, and where the row ends up.
struct WalkRow {
    bool map, in;    // a row of the map; a row at all
    int row;         // value row, or column of the map
    __device__ __forceinline__ WalkRow(const DeltaArgs &a, const Walk &w, int tid) {
        map = tid >= w.map_from;
        row = map ? tid - w.map_from : tid;
        in = map ? row < a.Dk : row < a.Dv;
    }
    __device__ __forceinline__ float *sum_out(const DeltaArgs &a, const Walk &w, int x) const {
        return map ? a.seg_map + (w.at * a.Dk + x) * a.Dk + row : a.seg_own + (w.at * a.Dk + x) * a.Dv + row;
    }
};

// What a walk's CTA sets up before its roles part; returns the tensor memory's base.
template <typename L>
__device__ __forceinline__ uint32_t walk_setup(WalkBars &bar, uint32_t sm32) {
    if (threadIdx.x == 0) {
        for (uint64_t *b : {&bar.full[0], &bar.full[1], &bar.empty[0], &bar.empty[1], &bar.rows[0], &bar.rows[1], &bar.rows[2], &bar.x, &bar.e, &bar.s,
                            &bar.o, &bar.g, &bar.drain[0], &bar.drain[1]})
            mbar_init(b, 1);
        *reinterpret_cast<volatile int *>(&bar.gone) = 0;
        bar.fetched = 0;
        fence_mbar_init();
    }
    // T and P are zero above the diagonal blocks, where prep never writes.
    for (uint32_t i = threadIdx.x; i < L::S * L::SLOT / 16; i += kWalkThreads) {
        const uint32_t z[4] = {0, 0, 0, 0};
        st_shared16(sm32 + L::T_AT + i * 16, z);
    }
    if (threadIdx.x < 32) tmem_alloc_all(&bar.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    return (uint32_t)warp_uniform((int)bar.tmem);
}

// First step of the it-th chunk that a walk comes to.
template <bool BWD>
__device__ __forceinline__ long long chunk_start(int it, int chunks) {
    return (long long)(BWD ? chunks - 1 - it : it) * DC;
}

// Sends for the rows of the it-th chunk (bfloat16); one thread of the walk, once the
// chunk KS before is done with.
template <typename L, bool BWD>
__device__ __forceinline__ void fetch_rows(const DeltaArgs &a, const CUtensorMap *kmap, const CUtensorMap *qmap, const CUtensorMap *vmap,
                                           WalkBars &bar, unsigned char *sm, const Seq &seq, int it, int chunks, int head) {
    if (it >= chunks) return;
    bar.fetched = it + 1;
    unsigned char *dst = sm + it % L::KS * L::ROWS;
    uint64_t *full = &bar.rows[it % L::KS];
    const int kh = head / (a.Hv / a.Hk), s = (int)(seq.s0 + chunk_start<BWD>(it, chunks)), b = (int)seq.b;
    // (The test hook makes CTA `stall_tile` expect 16 bytes that never come.)
    mbar_arrive_expect_tx(full, (2 * L::HALVES + (a.Dv > 64 ? 2 : 1)) * TILE + ((int)blockIdx.x == a.ctl.stall_tile ? 16 : 0));
#pragma unroll
    for (int h = 0; h < L::HALVES; ++h) {
        tma_load_4d(dst + h * 2 * TILE, kmap, h * 64, kh, s, b, full);
        tma_load_4d(dst + h * 2 * TILE + TILE, qmap, h * 64, kh, s, b, full);
    }
    for (int h = 0; h * 64 < a.Dv; ++h) tma_load_4d(dst + L::V_AT + h * TILE, vmap, h * 64, head, s, b, full);
    if (L::KS == 2 && it + 1 < chunks) {   // the next ones into L2 meanwhile
        const int s1 = (int)(seq.s0 + chunk_start<BWD>(it + 1, chunks));
#pragma unroll
        for (int h = 0; h < L::HALVES; ++h) {
            tma_prefetch_4d(kmap, h * 64, kh, s1, b);
            tma_prefetch_4d(qmap, h * 64, kh, s1, b);
        }
        for (int h = 0; h * 64 < a.Dv; ++h) tma_prefetch_4d(vmap, h * 64, head, s1, b);
    }
}

// End of a walk that gave up: the thread that issued the walk's products and copies waits
// for those in flight.
template <typename L>
__device__ __forceinline__ void drain_walk(WalkBars &bar, const Control &ctl) {
    drain_products(&bar.drain[0], ctl);
    if (L::KS > 1)
        for (int i = max(0, bar.fetched - L::KS); i < bar.fetched; ++i) drain_wait(&bar.rows[i % L::KS], (i / L::KS) & 1, ctl);
}

// The role of prep's threads (ptid 0 .. 255).  BWD: the backward's order and N.
template <typename T, int NT, int DK, int PT, bool BWD, bool RULE = true>
__device__ __forceinline__ void walk_prep(const DeltaArgs &a, const void *third, const qsh::Strides &st3, WalkBars &bar, unsigned char *sm,
                                          const Seq &seq, int chunks, int head, uint32_t tm, uint32_t gram_at) {
    using L = WalkLayout<NT, DK, PT>;
    const int ptid = threadIdx.x - 256, warp = warp_uniform(ptid / 32), kh = head / (a.Hv / a.Hk), half = ptid / 128;
    const uint32_t sm32 = smem_addr(sm);
    volatile int *gone = &bar.gone;
    bool ok = true;
    float *tf = reinterpret_cast<float *>(sm + L::F_AT);
    ChunkGates *gates = reinterpret_cast<ChunkGates *>(sm + L::GATES_AT);
    const uint32_t g_at = tm + ((uint32_t)(warp % 4 * 32) << 16) + gram_at;
    // Gram: rows 0-63 K K^T, rows 64-127 Q K^T, once the rows are there.
    auto gram = [&](int it) {
        const uint32_t rows = sm32 + it % L::KS * L::ROWS;
        if (NT == 1) {
            const int left = (int)min((long long)DC, seq.len - chunk_start<BWD>(it, chunks));
            // Rows past a packed sequence's end are another sequence's (past S, TMA fills with zeros).
            if (a.offsets && left < DC) {
                ok &= tc_wait_warp(&bar.rows[it % L::KS], (it / L::KS) & 1, gone, a.ctl);
                const uint32_t z[4] = {0, 0, 0, 0};
                for (int i = ptid; i < (DC - left) * 8; i += kPrepThreads) {
                    const uint32_t at = rows + (left + i / 8) * 128 + i % 8 * 16;
                    for (uint32_t tile = 0; tile < L::ROWS; tile += TILE) st_shared16(at + tile, z);
                }
                fence_proxy_async_smem();
                named_bar_sync(2, kPrepThreads);
            }
        }
        if (warp == 0 && elect_one()) {
            if (NT == 1) ok &= tc_wait(&bar.rows[it % L::KS], (it / L::KS) & 1, gone, a.ctl);
            tc_fence_after();
            if (ok) {
                const uint64_t kq = smem_desc(rows, 16, 1024);
                issue_ss<NT, NT, 2, DK / 16>(tm + gram_at, kq, L::KQ_TERM, kq, L::KQ_TERM, mma_desc(128, 64), KMajor(), KMajor());
                mma_commit(&bar.g);
            }
        }
        __syncwarp();
    };
    RawGates raw = {};
    if (warp == 7 && chunks > 0) {
        warp_gates(gates[0], read_gates<RULE>(a, seq, chunk_start<BWD>(0, chunks), head));
        if (chunks > 1) raw = read_gates<RULE>(a, seq, chunk_start<BWD>(1, chunks), head);
    }
    if (NT == 1 && chunks > 0) {
        named_bar_sync(2, kPrepThreads);
        gram(0);
    }
#pragma unroll 1
    for (int it = 0; it < chunks; ++it) {
        const ChunkGates &gt = gates[it & 3];
        const uint32_t slot = sm32 + L::T_AT + it % L::S * L::SLOT, p_at = slot + L::P_IN;
        if constexpr (NT == 3) {
            const long long t0 = chunk_start<BWD>(it, chunks);
            if (it > 0) ok &= tc_wait_warp(&bar.s, (it - 1) & 1, gone, a.ctl);   // the rows before are done with
            if (half == 0) load_rows<T, NT, DK, 128>(sm32, 2 * TILE, L::KQ_TERM, a.k, a.sk, seq, t0, kh, a.Dk, ptid);
            else load_rows<T, NT, DK, 128>(sm32 + TILE, 2 * TILE, L::KQ_TERM, a.q, a.sq, seq, t0, kh, a.Dk, ptid - 128);
            load_rows<T, NT, 128, kPrepThreads>(sm32 + L::V_AT, TILE, L::V_TERM, third, st3, seq, t0, head, a.Dv, ptid);
            fence_proxy_async_smem();
            named_bar_sync(2, kPrepThreads);
            gram(it);
        }
        ok &= tc_wait_warp(&bar.g, it & 1, gone, a.ctl);
        ok &= tc_wait_warp(&bar.empty[it % L::S], ((it / L::S) & 1) ^ 1, gone, a.ctl);   // the slot of T and P
        // A row of the Gram product per thread, the 16-column pieces p % 2 == half, with the
        // decays.  Below the warp's 32-row diagonal block D_ts = exp(G_t - G_31) exp(G_31 - G_s),
        // both at most one: no exp per value.
        {
            const int t = ptid % 64, wb = t / 32;
            const bool keys = ptid % 128 < 64;
            const Sum2 mine = gt.sum[t];
            const float row = wb ? decay(mine, gt.sum[31]) : 0.f, mul = keys ? (BWD ? gt.beta[t] : 1.f) : a.scale;
#pragma unroll 1
            for (int h = 0; h <= wb; ++h) {
                const int s0 = h * 32 + half * 16;
                uint32_t g[16];
                float x[16];
                __syncwarp();
                tmem_ld16(g_at + s0, g);
                if (h < wb) {
                    const float rm = row * mul;
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(&gt.mid[s0 + i]);
                        x[i] = m.x * rm, x[i + 1] = m.y * rm, x[i + 2] = m.z * rm, x[i + 3] = m.w * rm;
                    }
                } else {
                    const int last = keys ? t - 1 : t;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const Sum2 o = gt.sum[s0 + i];
                        const float d = exp2_fast(s0 + i <= t ? (mine.hi - o.hi) + (mine.lo - o.lo) : 0.f);
                        x[i] = s0 + i <= last ? d * mul : 0.f;
                    }
                }
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = x[i] == 0.f ? 0.f : x[i] * __uint_as_float(g[i]);   // (masked places stay 0)
                if (!RULE && keys) continue;   // (no T)
                if (keys) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        float4 be = make_float4(1.f, 1.f, 1.f, 1.f);
                        if (!BWD) be = *reinterpret_cast<const float4 *>(&gt.beta[s0 + i]);
                        store4(tf + t * FLD + s0 + i, make_float4(x[i] * be.x, x[i + 1] * be.y, x[i + 2] * be.z, x[i + 3] * be.w));
                    }
                } else {
                    store_terms<PT>(p_at, t, s0 / 8, x);
                    store_terms<PT>(p_at, t, s0 / 8 + 1, x + 8);
                }
            }
        }
        tc_fence_before();
        named_bar_sync(2, kPrepThreads);
        if (it + 1 < chunks) {   // the next chunk's gates and Gram products, under way while this one is inverted
            if (warp == 7) {
                warp_gates(gates[(it + 1) & 3], raw);
                if (it + 2 < chunks) raw = read_gates<RULE>(a, seq, chunk_start<BWD>(it + 2, chunks), head);
            }
            if (L::KS > 2) gram(it + 1);
        }
        if (RULE) {
            invert_64(tf, ptid, 2);
            store_inverse(slot, tf, ptid);
        }
        fence_proxy_async_smem();
        named_bar_sync(2, kPrepThreads);
        if (ptid == 0) mbar_arrive(&bar.full[it % L::S]);
        __syncwarp();
        if (L::KS == 2 && it + 1 < chunks) gram(it + 1);   // (its rows come only once the walk is a chunk further)
    }
    if (warp == 0 && elect_one() && (!ok || *gone)) drain_products(&bar.drain[1], a.ctl);
    __syncwarp();
}

// Sixteen values of the third tensor for value row dv, from step h on.
template <int NT>
__device__ __forceinline__ void third_column(const unsigned char *tiles, int dv, int h, float *v) {
    const unsigned char *p = tiles + dv / 64 * TILE + dv % 8 * 2 + h * 128;
    const uint32_t unit = (uint32_t)(dv % 64 / 8) << 4;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] = 0.f;
#pragma unroll
        for (int j = NT - 1; j >= 0; --j)
            v[i] += __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(p + j * 2 * TILE + i * 128 + (unit ^ (uint32_t)(i % 8 << 4))));
    }
}

// Stores sixteen steps of a value column per thread (the lanes of a warp hold 32 columns
// side by side) to rows `step` apart, as far as `left` goes; `out` points at the thread's own
// column.  bfloat16: four lanes trade their values first, so that each stores four columns
// of every fourth step (8 bytes; a 2-byte store per step costs four times the instructions).
// `in`: the thread's column exists (D is a multiple of 8: for four neighbours alike).
__device__ __forceinline__ void store_columns(float *out, size_t step, int left, bool in, const float *x) {
    if (in)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) out[i * step] = x[i];
    __syncwarp();
}
__device__ __forceinline__ void store_columns(__nv_bfloat16 *out, size_t step, int left, bool in, const float *x) {
    const int lane = threadIdx.x % 32, odd = lane & 1, far = lane >> 1 & 1, mine = odd + 2 * far;   // the step of four that this lane stores
    out += mine * step - lane % 4;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        // Two lanes: the even one gets both columns of steps i and i + 2, the odd one of i + 1 and i + 3.
        const uint32_t a = pack_bf16(x[i], x[i + 1]), b = pack_bf16(x[i + 2], x[i + 3]);
        const uint32_t oa = __shfl_xor_sync(0xffffffffu, a, 1), ob = __shfl_xor_sync(0xffffffffu, b, 1);
        const uint32_t p = odd ? __byte_perm(oa, a, 0x7632) : __byte_perm(a, oa, 0x5410);
        const uint32_t q = odd ? __byte_perm(ob, b, 0x7632) : __byte_perm(b, ob, 0x5410);
        // Then pairs of lanes: the first keeps the earlier step, the second the later one.
        const uint32_t o = __shfl_xor_sync(0xffffffffu, far ? p : q, 2);
        if (in && i + mine < left) *reinterpret_cast<uint2 *>(out + i * step) = far ? make_uint2(o, q) : make_uint2(p, o);
    }
    __syncwarp();
}

// Three terms of sixteen fp32 values, `term` columns apart, eight columns each.
__device__ __forceinline__ void put_terms3(uint32_t at, uint32_t term, const float2 *x) {
    uint32_t t[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t p[3];
        split2<3>(x[i], p);
        t[0][i] = p[0], t[1][i] = p[1], t[2][i] = p[2];
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) tmem_st8(at + j * term, t[j]);
}

}  // namespace qs
