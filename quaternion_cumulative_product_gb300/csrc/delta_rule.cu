// delta_rule.cu -- the gated delta rule over whole sequences: forward, and
// backward from the forward's carries and errors.
#include <cstring>

#include "delta_bwd_tc.cuh"
#include "delta_chain_tc.cuh"
#include "delta_fwd_tc.cuh"

namespace {

using namespace qs;

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

// A walk over the chunks, one CTA per (sequence, value head).  fp32 inputs take three
// times the space of K and Q: one stage.
template <bool BWD, typename T, int NT>
int launch_walks(const DeltaArgs &a, cudaStream_t stream) {
    constexpr int STAGES = NT == 1 ? 2 : 1, PT = BWD || NT == 3 ? 3 : 2;
    CUtensorMap maps[3];
    if (NT == 1 && a.B * a.S > 0) {
        const qsh::Strides so = {(long long)(a.S * a.Hv * a.Dv), (long long)a.Hv * a.Dv, a.Dv};
        int rc = qsh::head_map(&maps[0], a.k, a.sk, a.B, a.S, a.Hk, a.Dk);
        if (rc == QS_OK) rc = qsh::head_map(&maps[1], a.q, a.sq, a.B, a.S, a.Hk, a.Dk);
        if (rc == QS_OK) rc = BWD ? qsh::head_map(&maps[2], a.d_o, so, a.B, a.S, a.Hv, a.Dv)
                                  : qsh::head_map(&maps[2], a.v, a.sv, a.B, a.S, a.Hv, a.Dv);
        if (rc != QS_OK) return rc;
    }
    auto go = [&](auto kernel, size_t smem) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
            cudaGetLastError();
            return (int)QS_ERR_CUDA;
        }
        kernel<<<(unsigned)(a.N * a.Hv), kWalkThreads, smem, stream>>>(a, maps[0], maps[1], maps[2]);
        return launched();
    };
    constexpr size_t small = WalkLayout<NT, 64, STAGES, PT>::BYTES, large = WalkLayout<NT, 128, STAGES, PT>::BYTES;
    if constexpr (BWD) return a.Dk <= 64 ? go(delta_chain_tc_kernel<T, NT, 64, STAGES>, small) : go(delta_chain_tc_kernel<T, NT, 128, STAGES>, large);
    else return a.Dk <= 64 ? go(delta_fwd_tc_kernel<T, NT, 64, STAGES>, small) : go(delta_fwd_tc_kernel<T, NT, 128, STAGES>, large);
}

template <typename T, int NT, int CT>
int launch_chunks(const DeltaArgs &a, cudaStream_t stream) {
    auto go = [&](auto kernel, size_t smem) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
            cudaGetLastError();
            return (int)QS_ERR_CUDA;
        }
        kernel<<<(unsigned)(a.slots * a.Hv), kChunkThreads, smem, stream>>>(a);
        return launched();
    };
    return a.Dk <= 64 ? go(delta_chunk_tc_kernel<T, NT, CT, 64>, ChunkLayout<NT, CT, 64>::BYTES)
                      : go(delta_chunk_tc_kernel<T, NT, CT, 128>, ChunkLayout<NT, CT, 128>::BYTES);
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
    if (strides && (qsh::bad_strides(a.sq, es) || qsh::bad_strides(a.sk, es) || qsh::bad_strides(a.sv, es) ||
                    qsh::has_flat_dim(a.sq, B, S, Hk) || qsh::has_flat_dim(a.sk, B, S, Hk) || qsh::has_flat_dim(a.sv, B, S, Hv)))
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
    return dtype == QS_BF16 ? launch_walks<false, __nv_bfloat16, 1>(a, stream) : launch_walks<false, float, 3>(a, stream);
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
    if (strides && (qsh::bad_strides(a.sq, es) || qsh::bad_strides(a.sk, es) || qsh::bad_strides(a.sv, es) ||
                    qsh::has_flat_dim(a.sq, B, S, Hk) || qsh::has_flat_dim(a.sk, B, S, Hk) || qsh::has_flat_dim(a.sv, B, S, Hv)))
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
    a.ahead = (unsigned)sms;
    rc = dtype == QS_BF16 ? launch_walks<true, __nv_bfloat16, 1>(a, stream) : launch_walks<true, float, 3>(a, stream);
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
