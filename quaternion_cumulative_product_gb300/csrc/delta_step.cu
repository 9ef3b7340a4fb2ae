// delta_step.cu -- the gated delta rule for single tokens (or a few), on states
// that stay in a pool.
//
// Mathematics.  With a = exp(g), x = M^T k and y = M^T q of the old state M:
//     e = v - a x,   u = beta e,   M' = a M + k u^T,   o = scale (a y + <q, k> u),
// so both products with the state are taken in one read of it and one round of
// sums; the new state follows without a second pass.
//
// Bound: memory (the state is read and written once: 8 bytes a value against 7
// operations).  A CTA of 128 threads holds Dk x 32 values of one head's state in
// registers, 8 x 4 per thread at Dk = 128: eight 16-byte loads in flight per
// thread.  Splitting the value dimension over CTAs (rather than one CTA per
// head) is what fills the GPU when there are few sequences; a 32-value row is
// one full 128-byte line.
// Loads of a CTA that has come to its arithmetic leave memory idle, so each head's first
// CTA, its own loads under way, brings the state of a head that starts about when it ends
// to L2 (one bulk prefetch; as many heads ahead as there are SMs, half or twice that is the same).
// Measured, 256 sequences x 32 heads x 128 x 128: 171 us, 6.3 TB/s (93% of a copy's rate); without the
// prefetch 187 us, prefetch sent before the own loads 175; with four CTAs per SM (105
// registers) instead of five 188 and, without the prefetch, 205; six 197.  Streaming the
// state through shared memory with bulk copies took 188 to 236 us depending on the ring, whole
// rows per CTA 255.  A call for a single token of one sequence is a launch: 2.8 us on the device.
#include "mixer_device.cuh"
#include "quat_device.cuh"
#include "quat_host.h"
#include "quat_mixer.h"

namespace {

constexpr int kThreads = 128, kCols = 32, kRows = 8;   // rows of the state per thread, at most

struct StepArgs {
    const void *q, *k, *v, *g, *beta;
    float *state;
    const int *slots;
    void *o;
    qsh::Strides sq, sk, sv;
    long long P;
    int T, Hk, Hv, Dk, Dv;
    unsigned tiles;     // CTAs per head: value columns / 32
    unsigned ahead;     // heads between a CTA's own and the one whose state it brings to L2
    bool gate16;
    float scale;
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 5) delta_step_kernel(const StepArgs a) {
    __shared__ float part[2][4][3][kCols];   // [token parity][warp][x, y; <q,k>][column]
    const unsigned tile = blockIdx.x % a.tiles, head = (blockIdx.x / a.tiles) % a.Hv;
    const unsigned n = blockIdx.x / a.tiles / a.Hv;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int col = tile * kCols + (lane % 8) * 4;      // this thread's four columns
    const int rowg = warp * 4 + lane / 8;               // and its rows: rowg * R ..
    const int R = (a.Dk + 15) / 16, row0 = rowg * R;
    const bool in = col < a.Dv;
    const long long slot = a.slots ? a.slots[n] : (long long)n;
    const bool live = slot >= 0 && slot < a.P;
    T *o = static_cast<T *>(a.o) + (((size_t)n * a.T) * a.Hv + head) * a.Dv + col;
    if (!live) {   // the whole CTA takes this branch
        for (int t = 0; t < a.T; ++t)
            if (rowg == 0 && in) qs::store4(o + (size_t)t * a.Hv * a.Dv, qs::q_zero());
        return;
    }
    float *st = a.state + (((size_t)slot * a.Hv + head) * a.Dk + row0) * a.Dv + col;
    float4 m[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        m[i] = qs::q_zero();
        if (in && i < R && row0 + i < a.Dk) m[i] = *reinterpret_cast<const float4 *>(st + (size_t)i * a.Dv);
    }
    if (tile == 0 && threadIdx.x == 0) {
        const unsigned next = blockIdx.x / a.tiles + a.ahead;
        if (next < gridDim.x / a.tiles) {
            const long long its = a.slots ? a.slots[next / a.Hv] : (long long)(next / a.Hv);
            if (its >= 0 && its < a.P)
                qs::bulk_prefetch(a.state + ((size_t)its * a.Hv + next % a.Hv) * a.Dk * a.Dv, (uint32_t)(a.Dk * a.Dv) * 4);
        }
    }
    const unsigned kh = head / (a.Hv / a.Hk);
    const T *qp = static_cast<const T *>(a.q) + n * a.sq.b + kh * a.sq.h + row0;
    const T *kp = static_cast<const T *>(a.k) + n * a.sk.b + kh * a.sk.h + row0;
    const T *vp = static_cast<const T *>(a.v) + n * a.sv.b + head * a.sv.h + col;
    for (int t = 0; t < a.T; ++t) {
        float q[kRows], k[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const bool on = i < R && row0 + i < a.Dk;
            q[i] = on ? qs::load1(qp + (long long)t * a.sq.s + i) : 0.f;
            k[i] = on ? qs::load1(kp + (long long)t * a.sk.s + i) : 0.f;
        }
        const long long gi = ((long long)n * a.T + t) * a.Hv + head;
        const float alpha = expf(qs::load_any(a.g, a.gate16, gi)), beta = qs::load_any(a.beta, a.gate16, gi);
        const float4 v = in ? qs::load4(vp + (long long)t * a.sv.s) : qs::q_zero();
        float4 x = qs::q_zero(), y = qs::q_zero();
        float qk = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            x = make_float4(fmaf(k[i], m[i].x, x.x), fmaf(k[i], m[i].y, x.y), fmaf(k[i], m[i].z, x.z), fmaf(k[i], m[i].w, x.w));
            y = make_float4(fmaf(q[i], m[i].x, y.x), fmaf(q[i], m[i].y, y.y), fmaf(q[i], m[i].z, y.z), fmaf(q[i], m[i].w, y.w));
            qk = fmaf(q[i], k[i], qk);
        }
#pragma unroll
        for (int s = 8; s < 32; s *= 2) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, s);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, s);
            x.z += __shfl_xor_sync(0xffffffffu, x.z, s);
            x.w += __shfl_xor_sync(0xffffffffu, x.w, s);
            y.x += __shfl_xor_sync(0xffffffffu, y.x, s);
            y.y += __shfl_xor_sync(0xffffffffu, y.y, s);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, s);
            y.w += __shfl_xor_sync(0xffffffffu, y.w, s);
            qk += __shfl_xor_sync(0xffffffffu, qk, s);
        }
        float(*p)[3][kCols] = part[t & 1];
        if (lane < 8) {
            qs::store4(&p[warp][0][lane * 4], x);
            qs::store4(&p[warp][1][lane * 4], y);
            if (lane == 0) p[warp][2][0] = qk;
        }
        // One barrier per token: the other parity's sums were read before it.
        __syncthreads();
        x = y = qs::q_zero();
        qk = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float4 px = *reinterpret_cast<const float4 *>(&p[w][0][(lane % 8) * 4]);
            const float4 py = *reinterpret_cast<const float4 *>(&p[w][1][(lane % 8) * 4]);
            x = qs::q_add(x, px);
            y = qs::q_add(y, py);
            qk += p[w][2][0];
        }
        const float4 u = make_float4(beta * fmaf(-alpha, x.x, v.x), beta * fmaf(-alpha, x.y, v.y),
                                     beta * fmaf(-alpha, x.z, v.z), beta * fmaf(-alpha, x.w, v.w));
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            m[i] = make_float4(fmaf(alpha, m[i].x, k[i] * u.x), fmaf(alpha, m[i].y, k[i] * u.y),
                               fmaf(alpha, m[i].z, k[i] * u.z), fmaf(alpha, m[i].w, k[i] * u.w));
        if (rowg == 0 && in)
            qs::store4(o + (size_t)t * a.Hv * a.Dv,
                       make_float4(a.scale * fmaf(alpha, y.x, qk * u.x), a.scale * fmaf(alpha, y.y, qk * u.y),
                                   a.scale * fmaf(alpha, y.z, qk * u.z), a.scale * fmaf(alpha, y.w, qk * u.w)));
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
        if (in && i < R && row0 + i < a.Dk) qs::store4(st + (size_t)i * a.Dv, m[i]);
}

}  // namespace

extern "C" int quat_delta_step(int dtype, int gate_dtype, float scale, const void *q, const void *k, const void *v,
                               const void *g, const void *beta, float *state, const int32_t *slots, void *o,
                               const int64_t *strides, int64_t P, int64_t N, int64_t T, int64_t Hk, int64_t Hv, int64_t Dk,
                               int64_t Dv, void *stream_) {
    if ((dtype != QS_F32 && dtype != QS_BF16) || (gate_dtype != QS_F32 && gate_dtype != QS_BF16)) return QS_ERR_DIMS;
    if (P < 0 || N < 0 || T < 0 || Hk < 0 || Hv < 0 || Dk < 0 || Dv < 0) return QS_ERR_DIMS;
    const int64_t lim = int64_t(1) << 31;
    if (P >= lim || N >= lim || T >= lim || Hk >= lim || Hv >= lim) return QS_ERR_DIMS;
    if (Dk > QS_DELTA_MAX_D || Dv > QS_DELTA_MAX_D || Dk % 8 || Dv % 8) return QS_ERR_DIMS;
    if (Hv > 0 && (Hk == 0 || Hv % Hk)) return QS_ERR_DIMS;
    if (N == 0 || T == 0 || Hv == 0 || Dv == 0) return QS_OK;
    if (Dk == 0 || (!slots && N > P)) return QS_ERR_DIMS;
    const unsigned tiles = (unsigned)((Dv + kCols - 1) / kCols);
    if ((__int128)N * Hv * tiles >= lim || (__int128)N * T * Hv >= ((__int128)1 << 40)) return QS_ERR_DIMS;
    if (!q || !k || !v || !g || !beta || !o || (P && !state)) return QS_ERR_NULL;
    const int es = dtype == QS_BF16 ? 2 : 4, ge = gate_dtype == QS_BF16 ? 2 : 4;
    for (const void *p : {q, k, v, g, beta, (const void *)state, (const void *)slots, (const void *)o})
        if (qsh::misaligned(p)) return QS_ERR_MISALIGNED;
    StepArgs a{};
    a.sq = qsh::strides_of(strides, 0, T, Hk, Dk), a.sk = qsh::strides_of(strides, 1, T, Hk, Dk);
    a.sv = qsh::strides_of(strides, 2, T, Hv, Dv);
    if (strides && (qsh::bad_strides(a.sq, es) || qsh::bad_strides(a.sk, es) || qsh::bad_strides(a.sv, es)))
        return QS_ERR_MISALIGNED;
    const size_t gates = (size_t)N * T * Hv * ge, out = (size_t)N * T * Hv * Dv * es, pool = (size_t)P * Hv * Dk * Dv * 4;
    const struct { const void *p; size_t n; } ins[] = {
        {q, qsh::span_bytes(a.sq, N, T, Hk, Dk, es)}, {k, qsh::span_bytes(a.sk, N, T, Hk, Dk, es)},
        {v, qsh::span_bytes(a.sv, N, T, Hv, Dv, es)}, {g, gates}, {beta, gates}, {slots, (size_t)N * 4}};
    for (const auto &x : ins)
        if (qsh::overlaps(o, out, x.p, x.n) || qsh::overlaps(state, pool, x.p, x.n)) return QS_ERR_ALIAS;
    if (qsh::overlaps(o, out, state, pool)) return QS_ERR_ALIAS;
    int dev = 0, sms = 0;
    const int rc = qsh::device(&dev, &sms);
    if (rc != QS_OK) return rc;
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.state = state, a.slots = slots, a.o = o;
    a.P = P, a.T = (int)T, a.Hk = (int)Hk, a.Hv = (int)Hv, a.Dk = (int)Dk, a.Dv = (int)Dv, a.tiles = tiles, a.ahead = (unsigned)sms;
    a.gate16 = gate_dtype == QS_BF16, a.scale = scale;
    const unsigned grid = (unsigned)(N * Hv * tiles);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (dtype == QS_BF16) delta_step_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
    else delta_step_kernel<float><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? QS_OK : QS_ERR_CUDA;
}
