// norm_rotate.cu -- the per-head norm of queries and keys and their rotation by
// the conjugate of the cumulative quaternion, in one pass over memory, and its
// backward.
//
// Mathematics.  For a head vector x: r = (sum x^2 / div + eps)^(-1/2),
// n = x r w, z_j = conj(c_j) (x) n_j per quaternion.  Left multiplication by
// conj(c) is a 4x4 matrix whose transpose is left multiplication by c, so
//     dn_j = c_j (x) dz_j,      dc_j = n_j (x) conj(dz_j),
//     dw = sum over rows of dn x r,    dm = dn w,    dx = dm r - x r^3 <dm, x> / div.
// dc is summed over the query and key heads that share the rotation; one group
// of lanes handles all of them, so the sum stays in its registers.
//
// Bound: memory.  Every input is read once and every output written once, with
// 16-byte accesses where the head dimension allows them; the sums over a head
// are shuffles among the 1 .. 32 lanes that hold it (a power of two: 16 lanes of
// 8 values for D = 128).
// Measured: forward, 8 x 4096 x 16 heads of 128 bfloat16 with an fp32 cum, 115 us, 7.0 TB/s
// (the whole of a copy's rate).  The backward's figures are at kBwdCtasPerSm.
#include <mutex>

#include "mixer_device.cuh"
#include "quat_common.cuh"
#include "quat_host.h"
#include "quat_mixer.h"

namespace {

constexpr int kThreads = 256;

// CTAs per SM of the persistent backward, as many as run at once.  It issues about 330
// instructions per pair of rows and is bound by that, not by its loads: two CTAs of up
// to 128 registers (two quaternions per lane) take 82 us on 2 x 4099 rows of 32 + 8
// heads of 96, three of 80 registers 86 us, four with one quaternion per lane 89 us; a
// second row read ahead gains nothing.
constexpr int kBwdCtasPerSm = 2;

struct RotateArgs {
    const void *q, *k, *cum;
    const float *wq, *wk;
    const void *dqo, *dko;         // backward
    void *qo, *ko;                 // outputs (backward: d_q, d_k)
    void *dcum;
    float *dw_part;                // backward with weights: [CTAs][2][D]
    qsh::Strides sq, sk;
    unsigned S, H, J, D, nq, nk;   // nq, nk: heads per rotation
    unsigned items;                // B * S * H
    float eps, inv_div;
};

template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One group of LANES lanes per (step, rotation head); V quaternions per lane.
// SINGLE: one query and one key head per rotation (no loop, fewer registers).
template <typename T, typename C, int V, int LANES, bool SINGLE>
__global__ void __launch_bounds__(kThreads, SINGLE ? 6 : 4) rotate_fwd_kernel(const RotateArgs a) {
    const unsigned groups = kThreads / LANES;
    const unsigned item = blockIdx.x * groups + threadIdx.x / LANES;
    const unsigned lane = threadIdx.x % LANES, x0 = lane * V * 4;
    const bool live = item < a.items, in = live && x0 < a.D;
    const unsigned tok = live ? item / a.H : 0, h = live ? item - tok * a.H : 0;
    const unsigned b = tok / a.S, s = tok - b * a.S;

    float4 c[V];
    bool turn[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        turn[i] = in && lane * V + i < a.J;
        c[i] = qs::q_ident();
    }
    const C *cp = static_cast<const C *>(a.cum) + ((size_t)item * a.J + lane * V) * 4;
    if (turn[V - 1] && (V == 1 || a.J % 2 == 0 || sizeof(C) == 4)) qs::load_quads<V>(cp, c);
    else
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (turn[i]) c[i] = qs::load4(cp + 4 * i);

    const T *qp = static_cast<const T *>(a.q) + b * a.sq.b + s * a.sq.s + (long long)h * a.nq * a.sq.h + x0;
    const T *kp = static_cast<const T *>(a.k) + b * a.sk.b + s * a.sk.s + (long long)h * a.nk * a.sk.h + x0;
    T *qo = static_cast<T *>(a.qo) + (size_t)item * a.nq * a.D + x0;
    T *ko = static_cast<T *>(a.ko) + (size_t)item * a.nk * a.D + x0;

    auto row = [&](const float4 *x, const float *w, T *out) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += qs::dot4(x[i], x[i]);
        const float r = rsqrtf(fmaf(group_sum<LANES>(sum), a.inv_div, a.eps));
        float4 z[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float4 n = make_float4(x[i].x * r, x[i].y * r, x[i].z * r, x[i].w * r);
            if (w && in) {
                const float4 ww = qs::load4(w + x0 + 4 * i);
                n = make_float4(n.x * ww.x, n.y * ww.y, n.z * ww.z, n.w * ww.w);
            }
            z[i] = turn[i] ? qs::q_mul_cl(c[i], n) : n;
        }
        if (in) qs::store_quads<V>(out, z);
    };

    // The first query and key row are read together, the others of a shared
    // rotation one after the other (the loop's loads run ahead of its sums).
    float4 xq[V], xk[V];
#pragma unroll
    for (int i = 0; i < V; ++i) xq[i] = xk[i] = qs::q_zero();
    if (in && (SINGLE || a.nq)) qs::load_quads<V>(qp, xq);
    if (in && (SINGLE || a.nk)) qs::load_quads<V>(kp, xk);
    if constexpr (SINGLE) {
        row(xq, a.wq, qo);
        row(xk, a.wk, ko);
    } else {
        for (unsigned j = 0; j < a.nq; ++j) {
            float4 nx[V];
#pragma unroll
            for (int i = 0; i < V; ++i) nx[i] = qs::q_zero();
            if (in && j + 1 < a.nq) qs::load_quads<V>(qp + (j + 1) * a.sq.h, nx);
            row(xq, a.wq, qo + (size_t)j * a.D);
#pragma unroll
            for (int i = 0; i < V; ++i) xq[i] = nx[i];
        }
        for (unsigned j = 0; j < a.nk; ++j) {
            float4 nx[V];
#pragma unroll
            for (int i = 0; i < V; ++i) nx[i] = qs::q_zero();
            if (in && j + 1 < a.nk) qs::load_quads<V>(kp + (j + 1) * a.sk.h, nx);
            row(xk, a.wk, ko + (size_t)j * a.D);
#pragma unroll
            for (int i = 0; i < V; ++i) xk[i] = nx[i];
        }
    }
}

// Backward.  With weights the grid is persistent: each lane keeps its part of
// the weights' gradients in registers over all its rows, the CTA adds its
// groups up in a fixed order and writes one partial row, and
// rotate_weights_kernel adds the CTAs' partial rows up.
template <typename T, typename C, int V, int LANES, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, kBwdCtasPerSm) rotate_bwd_kernel(const RotateArgs a) {
    const unsigned groups = kThreads / LANES;
    const unsigned lane = threadIdx.x % LANES, x0 = lane * V * 4;
    const unsigned rounds = (a.items + gridDim.x * groups - 1) / (gridDim.x * groups);
    float4 dwq[V], dwk[V];
#pragma unroll
    for (int i = 0; i < V; ++i) dwq[i] = dwk[i] = qs::q_zero();

    for (unsigned it = 0; it < rounds; ++it) {
        const unsigned item = (it * gridDim.x + blockIdx.x) * groups + threadIdx.x / LANES;
        const bool live = item < a.items, in = live && x0 < a.D;
        const unsigned tok = live ? item / a.H : 0, h = live ? item - tok * a.H : 0;
        const unsigned b = tok / a.S, s = tok - b * a.S;
        float4 c[V], dc[V];
        bool turn[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            turn[i] = in && lane * V + i < a.J;
            c[i] = qs::q_ident();
            dc[i] = qs::q_zero();
        }
        const size_t cat = ((size_t)item * a.J + lane * V) * 4;
        const C *cp = static_cast<const C *>(a.cum) + cat;
        const bool wide = V == 1 || a.J % 2 == 0 || sizeof(C) == 4;
        if (turn[V - 1] && wide) qs::load_quads<V>(cp, c);
        else
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (turn[i]) c[i] = qs::load4(cp + 4 * i);

        // Lanes past the head read its start (their values count as zero).
        const unsigned at = in ? x0 : 0;
        auto rows = [&](const void *x_, const void *dz_, void *dx_, const qsh::Strides &st, unsigned n, const float *w,
                        float4 *dw) {
            const T *xp = static_cast<const T *>(x_) + b * st.b + s * st.s + (long long)h * n * st.h + at;
            const T *zp = static_cast<const T *>(dz_) + (size_t)(live ? item : 0) * n * a.D + at;
            T *op = static_cast<T *>(dx_) + (size_t)item * n * a.D + x0;
            float4 ww[V];
#pragma unroll
            for (int i = 0; i < V; ++i) ww[i] = WEIGHTS && w ? qs::load4(w + at + 4 * i) : make_float4(1.f, 1.f, 1.f, 1.f);
            qs::RawQuads<V, T> nx, nz;   // the next row, as it is in memory
            if (n) nx.load(xp), nz.load(zp);
            for (unsigned j = 0; j < n; ++j) {
                float4 x[V], dz[V];
                nx.get(x), nz.get(dz);
                if (j + 1 < n) nx.load(xp + (j + 1) * st.h), nz.load(zp + (size_t)(j + 1) * a.D);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (!in) x[i] = dz[i] = qs::q_zero();
                // <dm, x> and sum x^2 need no r: both sums run in one round of shuffles.
                float4 dn[V];
                float sum = 0.f, mix = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    dn[i] = turn[i] ? qs::q_mul(c[i], dz[i]) : dz[i];
                    sum += qs::dot4(x[i], x[i]);
                    mix += qs::dot4(make_float4(dn[i].x * ww[i].x, dn[i].y * ww[i].y, dn[i].z * ww[i].z, dn[i].w * ww[i].w), x[i]);
                }
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) {
                    sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    mix += __shfl_xor_sync(0xffffffffu, mix, o);
                }
                // (A group past the last item has no row: its r would be infinite without eps.  r^3 may be
                // past fp32 where r^3 <dm, x> x is not: r <dm, x> first.)
                const float r = live ? rsqrtf(fmaf(sum, a.inv_div, a.eps)) : 0.f;
                const float back = -(r * (r * (r * mix))) * a.inv_div;
                float4 dx[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float4 xr = make_float4(x[i].x * r, x[i].y * r, x[i].z * r, x[i].w * r);
                    if (turn[i]) {
                        const float4 n4 = make_float4(xr.x * ww[i].x, xr.y * ww[i].y, xr.z * ww[i].z, xr.w * ww[i].w);
                        dc[i] = qs::q_fma(dc[i], n4, qs::q_conj(dz[i]));
                    }
                    if (WEIGHTS && w)
                        dw[i] = make_float4(fmaf(dn[i].x, xr.x, dw[i].x), fmaf(dn[i].y, xr.y, dw[i].y),
                                            fmaf(dn[i].z, xr.z, dw[i].z), fmaf(dn[i].w, xr.w, dw[i].w));
                    dx[i] = make_float4(fmaf(x[i].x, back, dn[i].x * ww[i].x * r), fmaf(x[i].y, back, dn[i].y * ww[i].y * r),
                                        fmaf(x[i].z, back, dn[i].z * ww[i].z * r), fmaf(x[i].w, back, dn[i].w * ww[i].w * r));
                }
                if (in) qs::store_quads<V>(op + (size_t)j * a.D, dx);
            }
        };
        rows(a.q, a.dqo, a.qo, a.sq, a.nq, a.wq, dwq);
        rows(a.k, a.dko, a.ko, a.sk, a.nk, a.wk, dwk);
        C *dp = static_cast<C *>(a.dcum) + cat;
        if (turn[V - 1] && wide) qs::store_quads<V>(dp, dc);
        else
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (turn[i]) qs::store4(dp + 4 * i, dc[i]);
    }

    if constexpr (WEIGHTS) {
        __shared__ float part[kThreads * V * 4 * 2];   // [2][groups][LANES * V * 4]
        constexpr int W = LANES * V * 4;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            qs::store4(part + (threadIdx.x / LANES) * W + x0 + 4 * i, dwq[i]);
            qs::store4(part + (groups + threadIdx.x / LANES) * W + x0 + 4 * i, dwk[i]);
        }
        __syncthreads();
        for (unsigned x = threadIdx.x; x < 2 * a.D; x += kThreads) {
            const unsigned which = x / a.D, d = x - which * a.D;
            float sum = 0.f;
            for (unsigned gr = 0; gr < groups; ++gr) sum += part[(which * groups + gr) * W + d];
            a.dw_part[(size_t)blockIdx.x * 2 * a.D + x] = sum;
        }
    }
}

// d_w[x] = sum of the CTAs' partial rows: 32 strands of CTAs, each in order, then
// the strands in order.
__global__ void __launch_bounds__(1024) rotate_weights_kernel(const float *part, float *dwq, float *dwk, unsigned ctas, unsigned D) {
    __shared__ float strand[32][33];
    const unsigned x = blockIdx.x * 32 + threadIdx.x % 32, k = threadIdx.x / 32;
    float sum = 0.f;
    if (x < 2 * D)
#pragma unroll 4
        for (unsigned i = k; i < ctas; i += 32) sum += part[(size_t)i * 2 * D + x];
    strand[k][threadIdx.x % 32] = sum;
    __syncthreads();
    if (k == 0 && x < 2 * D) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) sum += strand[i][threadIdx.x];
        float *out = x < D ? dwq : dwk;
        if (out) out[x < D ? x : x - D] = sum;
    }
}

using Kernel = void (*)(RotateArgs);

// `FLAG`: with weights (backward), one head of either kind per rotation (forward).
template <bool BWD, bool FLAG, typename T, typename C, int V>
Kernel pick_lanes(int lanes) {
    auto one = [](auto l) -> Kernel {
        constexpr int L = decltype(l)::value;
        if constexpr (BWD) return rotate_bwd_kernel<T, C, V, L, FLAG>;
        else return rotate_fwd_kernel<T, C, V, L, FLAG>;
    };
    switch (lanes) {
        case 1: return one(std::integral_constant<int, 1>());
        case 2: return one(std::integral_constant<int, 2>());
        case 4: return one(std::integral_constant<int, 4>());
        case 8: return one(std::integral_constant<int, 8>());
        case 16: return one(std::integral_constant<int, 16>());
        default: return one(std::integral_constant<int, 32>());
    }
}

template <bool BWD, bool FLAG>
Kernel pick(int dtype, int cum_dtype, int v, int lanes) {
    using bf = __nv_bfloat16;
    if (dtype == QS_F32) {
        if (cum_dtype == QS_F32)
            return v == 2 ? pick_lanes<BWD, FLAG, float, float, 2>(lanes) : pick_lanes<BWD, FLAG, float, float, 1>(lanes);
        return v == 2 ? pick_lanes<BWD, FLAG, float, bf, 2>(lanes) : pick_lanes<BWD, FLAG, float, bf, 1>(lanes);
    }
    if (cum_dtype == QS_F32)
        return v == 2 ? pick_lanes<BWD, FLAG, bf, float, 2>(lanes) : pick_lanes<BWD, FLAG, bf, float, 1>(lanes);
    return v == 2 ? pick_lanes<BWD, FLAG, bf, bf, 2>(lanes) : pick_lanes<BWD, FLAG, bf, bf, 1>(lanes);
}

// Checks shared by the two directions: QS_OK, an error, or 1 for no rows at all.
int check(int dtype, int cum_dtype, int norm, float eps, int64_t B, int64_t S, int64_t H, int64_t J, int64_t Hq, int64_t Hk,
          int64_t D) {
    if ((dtype != QS_F32 && dtype != QS_BF16) || (cum_dtype != QS_F32 && cum_dtype != QS_BF16)) return QS_ERR_DIMS;
    if ((norm != QS_NORM_RMS && norm != QS_NORM_L2) || !(eps >= 0.f)) return QS_ERR_DIMS;
    if (B < 0 || S < 0 || H < 0 || J < 0 || Hq < 0 || Hk < 0 || D < 0) return QS_ERR_DIMS;
    const int64_t lim = int64_t(1) << 31;
    if (B >= lim || S >= lim || H >= lim || Hq >= lim || Hk >= lim || J >= lim) return QS_ERR_DIMS;
    if (D > QS_ROTATE_MAX_D || D % 4 || (D > 128 && D % 8) || 4 * J > D) return QS_ERR_DIMS;
    if (H > 0 && (Hq % H || Hk % H)) return QS_ERR_DIMS;
    if (H == 0 && (Hq || Hk)) return QS_ERR_DIMS;
    if ((__int128)B * S * H >= lim - kThreads || (__int128)B * S * (Hq > Hk ? Hq : Hk) >= lim) return QS_ERR_DIMS;
    return B * S * H == 0 || D == 0 || Hq + Hk == 0 ? 1 : QS_OK;
}

int lanes_of(int64_t D, int v) {
    int lanes = 1;
    while (lanes * v * 4 < D) lanes *= 2;
    return lanes;
}

int launched() {
    if (cudaGetLastError() != cudaSuccess) return QS_ERR_CUDA;
    return QS_OK;
}

}  // namespace

extern "C" int quat_norm_rotate_fwd(int dtype, int cum_dtype, int norm, float eps, const void *q, const void *k,
                                    const void *cum, const float *w_q, const float *w_k, void *q_out, void *k_out,
                                    const int64_t *strides, int64_t B, int64_t S, int64_t H, int64_t J, int64_t Hq,
                                    int64_t Hk, int64_t D, void *stream_) {
    const int dc = check(dtype, cum_dtype, norm, eps, B, S, H, J, Hq, Hk, D);
    if (dc == 1) return QS_OK;
    if (dc != QS_OK) return dc;
    if ((Hq && (!q || !q_out)) || (Hk && (!k || !k_out)) || (J && !cum)) return QS_ERR_NULL;
    const int es = dtype == QS_BF16 ? 2 : 4, cs = cum_dtype == QS_BF16 ? 2 : 4;
    const qsh::Strides sq = qsh::strides_of(strides, 0, S, Hq, D), sk = qsh::strides_of(strides, 1, S, Hk, D);
    for (const void *p : {q, k, cum, (const void *)w_q, (const void *)w_k, (const void *)q_out, (const void *)k_out})
        if (qsh::misaligned(p)) return QS_ERR_MISALIGNED;
    if (strides && ((Hq && qsh::bad_strides(sq, es)) || (Hk && qsh::bad_strides(sk, es)))) return QS_ERR_MISALIGNED;
    const size_t nq = (size_t)B * S * Hq * D * es, nk = (size_t)B * S * Hk * D * es, nc = (size_t)B * S * H * J * 4 * cs;
    const size_t iq = qsh::span_bytes(sq, B, S, Hq, D, es), ik = qsh::span_bytes(sk, B, S, Hk, D, es), nw = (size_t)D * 4;
    const struct { const void *p; size_t n; } ins[] = {{q, iq}, {k, ik}, {cum, nc}, {w_q, nw}, {w_k, nw}};
    for (const auto &i : ins)
        if (qsh::overlaps(q_out, nq, i.p, i.n) || qsh::overlaps(k_out, nk, i.p, i.n)) return QS_ERR_ALIAS;
    if (qsh::overlaps(q_out, nq, k_out, nk)) return QS_ERR_ALIAS;
    int dev = 0, sms = 0;
    const int rc = qsh::device(&dev, &sms);
    if (rc != QS_OK) return rc;
    RotateArgs a{};
    a.q = q, a.k = k, a.cum = cum, a.wq = w_q, a.wk = w_k, a.qo = q_out, a.ko = k_out, a.sq = sq, a.sk = sk;
    a.S = (unsigned)S, a.H = (unsigned)H, a.J = (unsigned)J, a.D = (unsigned)D;
    a.nq = (unsigned)(Hq / H), a.nk = (unsigned)(Hk / H), a.items = (unsigned)(B * S * H);
    a.eps = eps, a.inv_div = norm == QS_NORM_RMS ? 1.f / (float)D : 1.f;
    const int v = D % 8 == 0 ? 2 : 1, lanes = lanes_of(D, v), groups = kThreads / lanes;
    const Kernel fn = a.nq == 1 && a.nk == 1 ? pick<false, true>(dtype, cum_dtype, v, lanes) : pick<false, false>(dtype, cum_dtype, v, lanes);
    fn<<<(a.items + groups - 1) / groups, kThreads, 0, static_cast<cudaStream_t>(stream_)>>>(a);
    return launched();
}

extern "C" int quat_norm_rotate_bwd(int dtype, int cum_dtype, int norm, float eps, const void *q, const void *k,
                                    const void *cum, const float *w_q, const float *w_k, const void *d_q_out,
                                    const void *d_k_out, void *d_q, void *d_k, void *d_cum, float *d_w_q, float *d_w_k,
                                    const int64_t *strides, int64_t B, int64_t S, int64_t H, int64_t J, int64_t Hq,
                                    int64_t Hk, int64_t D, void *stream_) {
    const int dc = check(dtype, cum_dtype, norm, eps, B, S, H, J, Hq, Hk, D);
    if (dc != QS_OK && dc != 1) return dc;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if ((w_q && !d_w_q) || (w_k && !d_w_k)) return QS_ERR_NULL;
    if (qsh::misaligned(d_w_q) || qsh::misaligned(d_w_k)) return QS_ERR_MISALIGNED;
    if (dc == 1) {   // no rows: the sums over them are zero
        for (float *w : {w_q ? d_w_q : nullptr, w_k ? d_w_k : nullptr})
            if (w && D > 0 && cudaMemsetAsync(w, 0, (size_t)D * 4, stream) != cudaSuccess) {
                cudaGetLastError();
                return QS_ERR_CUDA;
            }
        if (B * S * H > 0 && D > 0 && J > 0) {   // rotations that no head uses
            if (!d_cum) return QS_ERR_NULL;
            if (cudaMemsetAsync(d_cum, 0, (size_t)B * S * H * J * 4 * (cum_dtype == QS_BF16 ? 2 : 4), stream) != cudaSuccess) {
                cudaGetLastError();
                return QS_ERR_CUDA;
            }
        }
        return QS_OK;
    }
    if ((Hq && (!q || !d_q || !d_q_out)) || (Hk && (!k || !d_k || !d_k_out)) || (J && (!cum || !d_cum))) return QS_ERR_NULL;
    const int es = dtype == QS_BF16 ? 2 : 4, cs = cum_dtype == QS_BF16 ? 2 : 4;
    const qsh::Strides sq = qsh::strides_of(strides, 0, S, Hq, D), sk = qsh::strides_of(strides, 1, S, Hk, D);
    for (const void *p : {q, k, cum, (const void *)w_q, (const void *)w_k, d_q_out, d_k_out, (const void *)d_q,
                          (const void *)d_k, (const void *)d_cum})
        if (qsh::misaligned(p)) return QS_ERR_MISALIGNED;
    if (strides && ((Hq && qsh::bad_strides(sq, es)) || (Hk && qsh::bad_strides(sk, es)))) return QS_ERR_MISALIGNED;
    const size_t nq = (size_t)B * S * Hq * D * es, nk = (size_t)B * S * Hk * D * es, nc = (size_t)B * S * H * J * 4 * cs;
    const size_t iq = qsh::span_bytes(sq, B, S, Hq, D, es), ik = qsh::span_bytes(sk, B, S, Hk, D, es), nw = (size_t)D * 4;
    const struct { const void *p; size_t n; } ins[] = {{q, iq}, {k, ik}, {cum, nc}, {w_q, nw}, {w_k, nw}, {d_q_out, nq}, {d_k_out, nk}};
    const struct { const void *p; size_t n; } outs[] = {{d_q, nq}, {d_k, nk}, {d_cum, nc}, {w_q ? d_w_q : nullptr, nw},
                                                        {w_k ? d_w_k : nullptr, nw}};
    for (int i = 0; i < 5; ++i) {
        for (const auto &x : ins)
            if (qsh::overlaps(outs[i].p, outs[i].n, x.p, x.n)) return QS_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (qsh::overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return QS_ERR_ALIAS;
    }
    int dev = 0, sms = 0;
    int rc = qsh::device(&dev, &sms);
    if (rc != QS_OK) return rc;
    RotateArgs a{};
    a.q = q, a.k = k, a.cum = cum, a.wq = w_q, a.wk = w_k, a.dqo = d_q_out, a.dko = d_k_out;
    a.qo = d_q, a.ko = d_k, a.dcum = d_cum, a.sq = sq, a.sk = sk;
    a.S = (unsigned)S, a.H = (unsigned)H, a.J = (unsigned)J, a.D = (unsigned)D;
    a.nq = (unsigned)(Hq / H), a.nk = (unsigned)(Hk / H), a.items = (unsigned)(B * S * H);
    a.eps = eps, a.inv_div = norm == QS_NORM_RMS ? 1.f / (float)D : 1.f;
    const int v = D % 8 == 0 ? 2 : 1, lanes = lanes_of(D, v), groups = kThreads / lanes;
    const unsigned all = (a.items + groups - 1) / groups;
    if (!w_q && !w_k) {
        pick<true, false>(dtype, cum_dtype, v, lanes)<<<all, kThreads, 0, stream>>>(a);
        return launched();
    }
    const unsigned most = (unsigned)(sms * kBwdCtasPerSm), grid = all < most ? all : most;
    unsigned char *ws = nullptr;
    qsh::Hold hold;
    rc = qsh::workspace(dev, stream, sizeof(qs::WsHeader) + (size_t)grid * 2 * D * 4, &ws, &hold);
    if (rc != QS_OK) return rc;
    a.dw_part = reinterpret_cast<float *>(ws + sizeof(qs::WsHeader));
    pick<true, true>(dtype, cum_dtype, v, lanes)<<<grid, kThreads, 0, stream>>>(a);
    rc = launched();
    if (rc != QS_OK) return rc;
    rotate_weights_kernel<<<(unsigned)(2 * D + 31) / 32, 1024, 0, stream>>>(a.dw_part, w_q ? d_w_q : nullptr,
                                                                          w_k ? d_w_k : nullptr, grid, (unsigned)D);
    return launched();
}
