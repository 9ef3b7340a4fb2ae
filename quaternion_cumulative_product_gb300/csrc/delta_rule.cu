// delta_rule.cu -- the gated delta rule over whole sequences: forward, and
// backward from the forward's carries and errors.
#include <cstring>

#include "delta_bwd_tc.cuh"
#include "delta_fwd_tc.cuh"

namespace {

using namespace qs;

constexpr int kThreads = 256;
constexpr int LD = QS_DELTA_MAX_D + 4, LC = DC + 1;   // padded rows in shared memory

// out(i, j, sum_k a(i, k) b(k, j)) over [M, N], K terms: 16 x 16 threads.
template <int M, int N, typename A, typename Bf, typename Out>
__device__ __forceinline__ void product(int K, const A &fa, const Bf &fb, const Out &out) {
    constexpr int TM = M / 16, TN = N / 16;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;
    for (int k = 0; k < K; ++k) {
        float x[TM], y[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) x[i] = fa(ty * TM + i, k);
#pragma unroll
        for (int j = 0; j < TN; ++j) y[j] = fb(k, tx + 16 * j);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) out(ty * TM + i, tx + 16 * j, acc[i][j]);
}

// Rows s .. s+63 of one head of a [B,S,H,D] tensor into dst [64][LD], zeros past
// the sequence and past D.
template <typename T>
__device__ __forceinline__ void load_tile(float (*dst)[LD], const void *p, const qsh::Strides &st, const Seq &seq, long long t0, int head, int D) {
    for (int i = threadIdx.x; i < DC * 128 / 4; i += kThreads) {
        const int t = i / 32, x = i % 32 * 4;
        float4 v = q_zero();
        if (t0 + t < seq.len && x < D)
            v = load4(static_cast<const T *>(p) + seq.b * st.b + (seq.s0 + t0 + t) * st.s + (long long)head * st.h + x);
        store4(&dst[t][x], v);
    }
}

struct Gates {
    Sum2 sum[DC];
    float beta[DC], grown[DC], left[DC];   // beta, exp(G_t), exp(G_C - G_t)
    float whole;                           // exp(G_C)
};

__device__ __forceinline__ void load_gates(Gates &s, const DeltaArgs &a, const Seq &seq, long long t0, int head) {
    if (threadIdx.x < 32) {
        float g[2], be[2];
        for (int i = 0; i < 2; ++i) {
            const long long t = t0 + 2 * threadIdx.x + i;
            const long long at = (seq.b * a.S + seq.s0 + t) * a.Hv + head;
            g[i] = t < seq.len ? clamp_gate(load_any(a.g, a.gate16, at)) : 0.f;
            be[i] = t < seq.len ? load_any(a.beta, a.gate16, at) : 0.f;
        }
        Sum2 s0, s1;
        chunk_sums(g[0], g[1], &s0, &s1);
        const Sum2 end = {__shfl_sync(0xffffffffu, s1.hi, 31), __shfl_sync(0xffffffffu, s1.lo, 31)};
        const int t = 2 * threadIdx.x;
        s.sum[t] = s0, s.sum[t + 1] = s1;
        s.beta[t] = be[0], s.beta[t + 1] = be[1];
        s.grown[t] = decay(s0, {0.f, 0.f}), s.grown[t + 1] = decay(s1, {0.f, 0.f});
        s.left[t] = decay(end, s0), s.left[t + 1] = decay(end, s1);
        if (threadIdx.x == 31) s.whole = s.grown[63];
    }
}

struct ChainSmem {
    float q[DC][LD], k[DC][LD], d[DC][LD], w[DC][LD];
    float a[DC][LC], p[DC][LC];
    Gates g;
};

// Backward, first kernel: one CTA per (sequence, value head) walks the chunks in
// reverse, writes dM' of every chunk and w.  The state's cotangent lives in the
// output array of the chunk before (in d_init's place in registers at the end).
template <typename T>
__global__ void __launch_bounds__(kThreads) delta_chain_simple_kernel(const DeltaArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    ChainSmem &s = *reinterpret_cast<ChainSmem *>(raw);
    const int head = blockIdx.x % a.Hv, kh = head / (a.Hv / a.Hk);
    const long long n = blockIdx.x / a.Hv;
    const Seq seq = seq_of(a, n);
    const size_t state = ((size_t)n * a.Hv + head) * a.Dk * a.Dv;
    const long long chunks = (seq.len + DC - 1) / DC;
    const qsh::Strides so = {(long long)a.S * a.Hv * a.Dv, (long long)a.Hv * a.Dv, a.Dv};
    float ds[8][8];   // rows ty*8+i, columns tx+16*j
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int i = 0; i < 8; ++i)
        for (int j = 0; j < 8; ++j) {
            const int x = ty * 8 + i, y = tx + 16 * j;
            ds[i][j] = a.d_final && x < a.Dk && y < a.Dv ? a.d_final[state + (size_t)x * a.Dv + y] : 0.f;
        }
    for (long long c = chunks - 1; c >= 0; --c) {
        const long long t0 = c * DC;
        float *out = a.ds + ((size_t)(seq.slot0 + c) * a.Hv + head) * a.Dk * a.Dv;
        for (int i = 0; i < 8; ++i)
            for (int j = 0; j < 8; ++j) {
                const int x = ty * 8 + i, y = tx + 16 * j;
                if (x < a.Dk && y < a.Dv) out[(size_t)x * a.Dv + y] = ds[i][j];
            }
        __syncthreads();
        load_tile<T>(s.q, a.q, a.sq, seq, t0, kh, a.Dk);
        load_tile<T>(s.k, a.k, a.sk, seq, t0, kh, a.Dk);
        load_tile<T>(s.d, a.d_o, so, seq, t0, head, a.Dv);
        load_gates(s.g, a, seq, t0, head);
        __syncthreads();
        auto gram = [&](float(*x)[LD], float(*o)[LC], bool diag, float f) {
            product<64, 64>(a.Dk, [&](int i, int k) { return x[i][k]; }, [&](int k, int j) { return s.k[j][k]; },
                            [&](int i, int j, float v) { o[i][j] = j < i || (diag && j == i) ? f * decay(s.g.sum[i], s.g.sum[j]) * v : 0.f; });
        };
        gram(s.k, s.a, false, 1.f);
        gram(s.q, s.p, true, a.scale);
        product<64, 128>(a.Dk, [&](int i, int k) { return s.k[i][k]; },
                         [&](int k, int j) { return j < a.Dv ? out[(size_t)k * a.Dv + j] : 0.f; },
                         [&](int i, int j, float v) { s.w[i][j] = s.g.left[i] * v; });
        __syncthreads();
        product<64, 128>(DC, [&](int i, int k) { return s.p[k][i]; }, [&](int k, int j) { return s.d[k][j]; },
                         [&](int i, int j, float v) { s.w[i][j] += v; });
        __syncthreads();
        if (threadIdx.x < 128) {
            for (int t = DC - 2; t >= 0; --t) {
                float w = s.w[t][threadIdx.x];
                for (int r = t + 1; r < DC; ++r) w = fmaf(-s.a[r][t] * s.g.beta[r], s.w[r][threadIdx.x], w);
                s.w[t][threadIdx.x] = w;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < DC * a.Dv; i += kThreads) {
            const int t = i / a.Dv, y = i % a.Dv;
            if (t0 + t < seq.len) {
                const size_t at = ((size_t)(seq.b * a.S + seq.s0 + t0 + t) * a.Hv + head) * a.Dv + y;
                a.w[at] = s.w[t][y];
                store1(static_cast<T *>(a.dv) + at, s.g.beta[t] * s.w[t][y]);
            }
        }
        float nd[8][8];
        product<128, 128>(DC, [&](int i, int k) { return s.g.grown[k] * a.scale * s.q[k][i]; }, [&](int k, int j) { return s.d[k][j]; },
                          [&](int i, int j, float v) { nd[i % 8][j / 16] = v; });
        product<128, 128>(DC, [&](int i, int k) { return s.g.grown[k] * s.g.beta[k] * s.k[k][i]; }, [&](int k, int j) { return s.w[k][j]; },
                          [&](int i, int j, float v) { ds[i % 8][j / 16] = fmaf(s.g.whole, ds[i % 8][j / 16], nd[i % 8][j / 16] - v); });
    }
    if (a.d_init)
        for (int i = 0; i < 8; ++i)
            for (int j = 0; j < 8; ++j) {
                const int x = ty * 8 + i, y = tx + 16 * j;
                if (x < a.Dk && y < a.Dv) a.d_init[state + (size_t)x * a.Dv + y] = ds[i][j];
            }
}

// dq, dk of a key head: the sum over the value heads that share it.
template <typename T>
__global__ void __launch_bounds__(256) delta_shared_kernel(const DeltaArgs a, long long quads) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= quads) return;
    const int dq = a.Dk / 4, G = a.Hv / a.Hk;
    const long long row = i / dq / a.Hk;
    const int x = (int)(i % dq) * 4, h = (int)(i / dq % a.Hk);
    float4 q = q_zero(), k = q_zero();
    for (int j = 0; j < G; ++j) {
        const size_t at = ((size_t)row * a.Hv + h * G + j) * a.Dk + x;
        q = q_add(q, load4(a.dqh + at));
        k = q_add(k, load4(a.dkh + at));
    }
    const size_t out = ((size_t)row * a.Hk + h) * a.Dk + x;
    store4(static_cast<T *>(a.dq) + out, q);
    store4(static_cast<T *>(a.dk) + out, k);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
int launched() { return cudaGetLastError() == cudaSuccess ? QS_OK : QS_ERR_CUDA; }

// Launches a walk kernel with its shared memory.
template <typename K>
int launch_walk(K kernel, const DeltaArgs &a, unsigned grid, unsigned threads, size_t smem, cudaStream_t stream) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
        cudaGetLastError();
        return QS_ERR_CUDA;
    }
    kernel<<<grid, threads, smem, stream>>>(a);
    return launched();
}

template <typename T, int NT>
int launch_fwd(const DeltaArgs &a, cudaStream_t stream) {
    constexpr int STAGES = NT == 1 ? 2 : 1;
    const unsigned grid = (unsigned)(a.N * a.Hv);
    if (a.Dk <= 64)
        return launch_walk(delta_fwd_tc_kernel<T, NT, 64, STAGES>, a, grid, kWalkThreads, WalkLayout<T, NT, 64, STAGES>::BYTES, stream);
    return launch_walk(delta_fwd_tc_kernel<T, NT, 128, STAGES>, a, grid, kWalkThreads, WalkLayout<T, NT, 128, STAGES>::BYTES, stream);
}

template <typename T, int NT, int CT>
int launch_chunks(const DeltaArgs &a, cudaStream_t stream) {
    const unsigned grid = (unsigned)(a.slots * a.Hv);
    if (a.Dk <= 64)
        return launch_walk(delta_chunk_tc_kernel<T, NT, CT, 64>, a, grid, kChunkThreads, ChunkLayout<NT, CT, 64>::BYTES, stream);
    return launch_walk(delta_chunk_tc_kernel<T, NT, CT, 128>, a, grid, kChunkThreads, ChunkLayout<NT, CT, 128>::BYTES, stream);
}

template <typename S, typename K>
int launch(K kernel, const DeltaArgs &a, unsigned grid, cudaStream_t stream) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(S)) != cudaSuccess) {
        cudaGetLastError();
        return QS_ERR_CUDA;
    }
    kernel<<<grid, kThreads, sizeof(S), stream>>>(a);
    return launched();
}

// Checks of sizes: QS_OK, an error, or 1 when there are no steps.
int check(int dtype, int gate_dtype, const int32_t *offsets, int64_t N, int64_t B, int64_t S, int64_t Hk, int64_t Hv,
          int64_t Dk, int64_t Dv) {
    if ((dtype != QS_F32 && dtype != QS_BF16) || (gate_dtype != QS_F32 && gate_dtype != QS_BF16)) return QS_ERR_DIMS;
    if (N < 0 || B < 0 || S < 0 || Hk < 0 || Hv < 0 || Dk < 0 || Dv < 0) return QS_ERR_DIMS;
    const int64_t lim = int64_t(1) << 31;
    if (N >= lim || B >= lim || S >= lim || Hk >= lim || Hv >= lim) return QS_ERR_DIMS;
    if (Dk > QS_DELTA_MAX_D || Dv > QS_DELTA_MAX_D || Dk % 8 || Dv % 8) return QS_ERR_DIMS;
    if (Hv > 0 && (Hk == 0 || Hv % Hk || Dk == 0 || Dv == 0)) return QS_ERR_DIMS;
    if (offsets ? B != 1 : N != B) return QS_ERR_DIMS;
    const int64_t slots = offsets ? S / DC + N : N * ((S + DC - 1) / DC);
    if ((__int128)N * Hv >= lim || (__int128)slots * Hv >= lim || (__int128)B * S * Hv >= ((__int128)1 << 40)) return QS_ERR_DIMS;
    return N * Hv == 0 ? 1 : QS_OK;
}

struct Sized {
    const void *p;
    size_t n;
};

int check_alias(const Sized *ins, int ni, const Sized *outs, int no) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (qsh::overlaps(outs[i].p, outs[i].n, ins[j].p, ins[j].n)) return QS_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (qsh::overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return QS_ERR_ALIAS;
    }
    return QS_OK;
}

void geometry(DeltaArgs &a, const int64_t *strides, const int32_t *offsets, int64_t N, int64_t B, int64_t S, int64_t Hk,
              int64_t Hv, int64_t Dk, int64_t Dv, int gate_dtype, float scale) {
    a.sq = qsh::strides_of(strides, 0, S, Hk, Dk), a.sk = qsh::strides_of(strides, 1, S, Hk, Dk);
    a.sv = qsh::strides_of(strides, 2, S, Hv, Dv);
    a.offsets = offsets, a.B = B, a.S = S, a.N = N, a.NC = (S + DC - 1) / DC;
    a.slots = offsets ? S / DC + N : N * a.NC;
    a.Hk = (int)Hk, a.Hv = (int)Hv, a.Dk = (int)Dk, a.Dv = (int)Dv;
    a.gate16 = gate_dtype == QS_BF16, a.scale = scale;
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

extern "C" int quat_delta_fwd(int dtype, int gate_dtype, float scale, const void *q, const void *k, const void *v,
                              const void *g, const void *beta, const float *init, void *o, float *final_state,
                              float *carries, float *errors, const int64_t *strides, const int32_t *offsets, int64_t N,
                              int64_t B, int64_t S, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, void *stream_) {
    const int dc = check(dtype, gate_dtype, offsets, N, B, S, Hk, Hv, Dk, Dv);
    if (dc == 1) return QS_OK;
    if (dc != QS_OK) return dc;
    const bool some = B * S > 0;
    if (some && (!q || !k || !v || !g || !beta || !o)) return QS_ERR_NULL;
    if (some && (carries == nullptr) != (errors == nullptr)) return QS_ERR_NULL;
    for (const void *p : {q, k, v, g, beta, (const void *)init, (const void *)o, (const void *)final_state,
                          (const void *)carries, (const void *)errors, (const void *)offsets})
        if (qsh::misaligned(p)) return QS_ERR_MISALIGNED;
    const int es = dtype == QS_BF16 ? 2 : 4, ge = gate_dtype == QS_BF16 ? 2 : 4;
    DeltaArgs a{};
    geometry(a, strides, offsets, N, B, S, Hk, Hv, Dk, Dv, gate_dtype, scale);
    if (strides && (qsh::bad_strides(a.sq, es) || qsh::bad_strides(a.sk, es) || qsh::bad_strides(a.sv, es)))
        return QS_ERR_MISALIGNED;
    const size_t gates = (size_t)B * S * Hv * ge, states = (size_t)N * Hv * Dk * Dv * 4, rows = (size_t)B * S * Hv * Dv;
    const Sized ins[] = {{q, qsh::span_bytes(a.sq, B, S, Hk, Dk, es)}, {k, qsh::span_bytes(a.sk, B, S, Hk, Dk, es)},
                         {v, qsh::span_bytes(a.sv, B, S, Hv, Dv, es)}, {g, gates}, {beta, gates}, {init, states},
                         {offsets, (size_t)(N + 1) * 4}};
    const Sized outs[] = {{o, rows * es}, {final_state, states}, {carries, (size_t)a.slots * Hv * Dk * Dv * 4}, {errors, rows * 4}};
    if (check_alias(ins, 7, outs, 4) != QS_OK) return QS_ERR_ALIAS;
    int dev = 0, sms = 0;
    const int rc = qsh::device(&dev, &sms);
    if (rc != QS_OK) return rc;
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.init = init, a.o = o, a.fin = final_state;
    a.carries = carries, a.errors = errors;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    unsigned char *ws = nullptr;
    const int wc = qsh::workspace(dev, stream, sizeof(WsHeader), &ws);
    if (wc != QS_OK) return wc;
    a.ctl = {reinterpret_cast<WsHeader *>(ws), -1, qsh::timeout_ns()};
    return dtype == QS_BF16 ? launch_fwd<__nv_bfloat16, 1>(a, stream) : launch_fwd<float, 3>(a, stream);
}

extern "C" int quat_delta_bwd(int dtype, int gate_dtype, float scale, const void *q, const void *k, const void *v,
                              const void *g, const void *beta, const float *carries, const float *errors, const void *d_o,
                              const float *d_final, void *d_q, void *d_k, void *d_v, void *d_g, void *d_beta, float *d_init,
                              const int64_t *strides, const int32_t *offsets, int64_t N, int64_t B, int64_t S, int64_t Hk,
                              int64_t Hv, int64_t Dk, int64_t Dv, void *stream_) {
    const int dc = check(dtype, gate_dtype, offsets, N, B, S, Hk, Hv, Dk, Dv);
    if (dc == 1) return QS_OK;
    if (dc != QS_OK) return dc;
    const bool some = B * S > 0;
    if (some && (!q || !k || !v || !g || !beta || !carries || !errors || !d_o || !d_q || !d_k || !d_v || !d_g || !d_beta))
        return QS_ERR_NULL;
    for (const void *p : {q, k, v, g, beta, (const void *)carries, (const void *)errors, d_o, (const void *)d_final,
                          (const void *)d_q, (const void *)d_k, (const void *)d_v, (const void *)d_g, (const void *)d_beta,
                          (const void *)d_init, (const void *)offsets})
        if (qsh::misaligned(p)) return QS_ERR_MISALIGNED;
    const int es = dtype == QS_BF16 ? 2 : 4, ge = gate_dtype == QS_BF16 ? 2 : 4;
    DeltaArgs a{};
    geometry(a, strides, offsets, N, B, S, Hk, Hv, Dk, Dv, gate_dtype, scale);
    if (strides && (qsh::bad_strides(a.sq, es) || qsh::bad_strides(a.sk, es) || qsh::bad_strides(a.sv, es)))
        return QS_ERR_MISALIGNED;
    const size_t gates = (size_t)B * S * Hv * ge, states = (size_t)N * Hv * Dk * Dv * 4, rows = (size_t)B * S * Hv * Dv;
    const size_t keys = (size_t)B * S * Hk * Dk, kept = (size_t)a.slots * Hv * Dk * Dv;
    const Sized ins[] = {{q, qsh::span_bytes(a.sq, B, S, Hk, Dk, es)}, {k, qsh::span_bytes(a.sk, B, S, Hk, Dk, es)},
                         {v, qsh::span_bytes(a.sv, B, S, Hv, Dv, es)}, {g, gates}, {beta, gates}, {carries, kept * 4},
                         {errors, rows * 4}, {d_o, rows * es}, {d_final, states}, {offsets, (size_t)(N + 1) * 4}};
    const Sized outs[] = {{d_q, keys * es}, {d_k, keys * es}, {d_v, rows * es}, {d_g, gates}, {d_beta, gates}, {d_init, states}};
    if (check_alias(ins, 10, outs, 6) != QS_OK) return QS_ERR_ALIAS;
    int dev = 0, sms = 0;
    int rc = qsh::device(&dev, &sms);
    if (rc != QS_OK) return rc;
    const bool shared = Hv != Hk;
    const size_t nds = align256(kept * 4), nw = align256(rows * 4), nh = shared ? align256((size_t)B * S * Hv * Dk * 4) : 0;
    unsigned char *ws = nullptr;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    rc = qsh::workspace(dev, stream, sizeof(WsHeader) + nds + nw + 2 * nh, &ws);
    if (rc != QS_OK) return rc;
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.carries_in = carries, a.errors_in = errors, a.d_o = d_o;
    a.d_final = d_final, a.dq = d_q, a.dk = d_k, a.dv = d_v, a.dg = d_g, a.dbeta = d_beta, a.d_init = d_init;
    unsigned char *p = ws + sizeof(WsHeader);
    a.ds = reinterpret_cast<float *>(p), a.w = reinterpret_cast<float *>(p + nds);
    a.dqh = reinterpret_cast<float *>(p + nds + nw), a.dkh = reinterpret_cast<float *>(p + nds + nw + nh);
    a.ctl = {reinterpret_cast<WsHeader *>(ws), -1, qsh::timeout_ns()};
    const unsigned chains = (unsigned)(N * Hv);
    rc = dtype == QS_BF16 ? launch<ChainSmem>(delta_chain_simple_kernel<__nv_bfloat16>, a, chains, stream)
                          : launch<ChainSmem>(delta_chain_simple_kernel<float>, a, chains, stream);
    if (rc != QS_OK || !some) return rc;
    if (dtype != QS_BF16) rc = launch_chunks<float, 3, 3>(a, stream);
    else rc = gate_dtype == QS_BF16 ? launch_chunks<__nv_bfloat16, 1, 2>(a, stream) : launch_chunks<__nv_bfloat16, 1, 3>(a, stream);
    if (rc != QS_OK || !shared) return rc;
    const long long quads = B * S * Hk * Dk / 4;
    const unsigned grid = (unsigned)((quads + 255) / 256);
    if (dtype == QS_BF16) delta_shared_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, quads);
    else delta_shared_kernel<float><<<grid, 256, 0, stream>>>(a, quads);
    return launched();
}
