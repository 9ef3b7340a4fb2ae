// decay.cu -- linear attention with a decay for each head over whole sequences: forward and
// backward.
//
// Mathematics: the delta rule's chunked form (delta_common.cuh) with e_t = v_t and beta = 1,
// so that no step of a chunk waits for another.
#include "delta_host.cuh"

using namespace qs;

extern "C" int quat_decay_fwd(int dtype, int gate_dtype, float scale, const void *q, const void *k, const void *v, const void *g,
                              const float *init, void *o, float *final_state, const int64_t *strides, const int32_t *offsets,
                              int64_t N, int64_t B, int64_t S, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, void *stream_) {
    const int dc = check(dtype, gate_dtype, offsets, N, B, S, Hk, Hv, Dk, Dv);
    if (dc == 1) return QS_OK;
    if (dc != QS_OK) return dc;
    const bool some = B * S > 0;
    if (some && (!q || !k || !v || !g || !o)) return QS_ERR_NULL;
    for (const void *p : {q, k, v, g, (const void *)init, (const void *)o, (const void *)final_state, (const void *)offsets})
        if (qsh::misaligned(p)) return QS_ERR_MISALIGNED;
    const int es = dtype == QS_BF16 ? 2 : 4, ge = gate_dtype == QS_BF16 ? 2 : 4;
    DeltaArgs a{};
    geometry(a, strides, offsets, N, B, S, Hk, Hv, Dk, Dv, gate_dtype, scale);
    if (strides && bad_layout(a, dtype)) return QS_ERR_MISALIGNED;
    const size_t gates = (size_t)B * S * Hv * ge, states = (size_t)N * Hv * Dk * Dv * 4, rows = (size_t)B * S * Hv * Dv;
    const Sized ins[] = {{q, qsh::span_bytes(a.sq, B, S, Hk, Dk, es)}, {k, qsh::span_bytes(a.sk, B, S, Hk, Dk, es)},
                         {v, qsh::span_bytes(a.sv, B, S, Hv, Dv, es)}, {g, gates}, {init, states}, {offsets, (size_t)(N + 1) * 4}};
    const Sized outs[] = {{o, rows * es}, {final_state, states}};
    if (check_alias(ins, 6, outs, 2) != QS_OK) return QS_ERR_ALIAS;
    int dev = 0, sms = 0;
    const int rc = qsh::device(&dev, &sms);
    if (rc != QS_OK) return rc;
    a.q = q, a.k = k, a.v = v, a.g = g, a.init = init, a.o = o, a.fin = final_state;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    unsigned char *ws = nullptr;
    cut(a, sms);
    qsh::Hold hold;
    const int wc = qsh::workspace(dev, stream, sizeof(WsHeader) + seg_floats(a) * 4, &ws, &hold);
    if (wc != QS_OK) return wc;
    float *seg = reinterpret_cast<float *>(ws + sizeof(WsHeader));
    a.ctl = {reinterpret_cast<WsHeader *>(ws), qsh::stall_tile(), qsh::timeout_ns()};
    return dtype == QS_BF16 ? launch_walks<false, __nv_bfloat16, 1, false>(a, seg, stream)
                            : launch_walks<false, float, 3, false>(a, seg, stream);
}

extern "C" int quat_decay_bwd(int dtype, int gate_dtype, float scale, const void *q, const void *k, const void *v, const void *g,
                              const float *init, const void *d_o, const float *d_final, void *d_q, void *d_k, void *d_v,
                              void *d_g, float *d_init, const int64_t *strides, const int32_t *offsets, int64_t N, int64_t B,
                              int64_t S, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, void *stream_) {
    const int dc = check(dtype, gate_dtype, offsets, N, B, S, Hk, Hv, Dk, Dv);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (dc == 1) {   // keys that no value head uses have zero gradients
        const size_t bytes = (size_t)B * S * Hk * Dk * (dtype == QS_BF16 ? 2 : 4);
        for (void *p : {d_q, d_k}) {
            if (bytes == 0) break;
            if (!p) return QS_ERR_NULL;
            if (cudaMemsetAsync(p, 0, bytes, stream) != cudaSuccess) {
                cudaGetLastError();
                return QS_ERR_CUDA;
            }
        }
        return QS_OK;
    }
    if (dc != QS_OK) return dc;
    const bool some = B * S > 0;
    if (some && (!q || !k || !v || !g || !d_o || !d_q || !d_k || !d_v || !d_g)) return QS_ERR_NULL;
    for (const void *p : {q, k, v, g, (const void *)init, d_o, (const void *)d_final, (const void *)d_q, (const void *)d_k,
                          (const void *)d_v, (const void *)d_g, (const void *)d_init, (const void *)offsets})
        if (qsh::misaligned(p)) return QS_ERR_MISALIGNED;
    const int es = dtype == QS_BF16 ? 2 : 4, ge = gate_dtype == QS_BF16 ? 2 : 4;
    DeltaArgs a{};
    geometry(a, strides, offsets, N, B, S, Hk, Hv, Dk, Dv, gate_dtype, scale);
    if (strides && bad_layout(a, dtype)) return QS_ERR_MISALIGNED;
    const size_t gates = (size_t)B * S * Hv * ge, states = (size_t)N * Hv * Dk * Dv * 4, rows = (size_t)B * S * Hv * Dv;
    const size_t keys = (size_t)B * S * Hk * Dk, kept = (size_t)a.slots * Hv * Dk * Dv;
    const Sized ins[] = {{q, qsh::span_bytes(a.sq, B, S, Hk, Dk, es)}, {k, qsh::span_bytes(a.sk, B, S, Hk, Dk, es)},
                         {v, qsh::span_bytes(a.sv, B, S, Hv, Dv, es)}, {g, gates}, {init, states}, {d_o, rows * es},
                         {d_final, states}, {offsets, (size_t)(N + 1) * 4}};
    const Sized outs[] = {{d_q, keys * es}, {d_k, keys * es}, {d_v, rows * es}, {d_g, gates}, {d_init, states}};
    if (check_alias(ins, 8, outs, 5) != QS_OK) return QS_ERR_ALIAS;
    int dev = 0, sms = 0;
    int rc = qsh::device(&dev, &sms);
    if (rc != QS_OK) return rc;
    const bool shared = Hv != Hk;
    const size_t nds = align256(kept * 4), nh = shared ? align256((size_t)B * S * Hv * Dk * 4) : 0;
    unsigned char *ws = nullptr;
    cut(a, sms);
    qsh::Hold hold;
    rc = qsh::workspace(dev, stream, sizeof(WsHeader) + 2 * nds + 2 * nh + seg_floats(a) * 4, &ws, &hold);
    if (rc != QS_OK) return rc;
    unsigned char *p = ws + sizeof(WsHeader);
    a.q = q, a.k = k, a.v = v, a.g = g, a.init = init, a.d_o = d_o, a.d_final = d_final;
    a.dq = d_q, a.dk = d_k, a.dv = d_v, a.dg = d_g, a.d_init = d_init;
    a.carries = reinterpret_cast<float *>(p), a.carries_in = a.carries;
    a.ds = reinterpret_cast<float *>(p + nds);
    a.dqh = reinterpret_cast<float *>(p + 2 * nds), a.dkh = reinterpret_cast<float *>(p + 2 * nds + nh);
    a.ctl = {reinterpret_cast<WsHeader *>(ws), qsh::stall_tile(), qsh::timeout_ns()};
    float *seg = reinterpret_cast<float *>(p + 2 * nds + 2 * nh);
    if (some)   // the states that enter the chunks
        rc = dtype == QS_BF16 ? launch_walks<false, __nv_bfloat16, 1, false>(a, seg, stream)
                              : launch_walks<false, float, 3, false>(a, seg, stream);
    if (rc != QS_OK) return rc;
    rc = dtype == QS_BF16 ? launch_walks<true, __nv_bfloat16, 1, false>(a, seg, stream)
                          : launch_walks<true, float, 3, false>(a, seg, stream);
    if (rc != QS_OK || !some) return rc;
    if (dtype != QS_BF16) rc = launch_chunks<float, 3, 3, false>(a, stream);
    else rc = gate_dtype == QS_BF16 ? launch_chunks<__nv_bfloat16, 1, 2, false>(a, stream) : launch_chunks<__nv_bfloat16, 1, 3, false>(a, stream);
    if (rc != QS_OK || !shared) return rc;
    const long long quads = B * S * Hk * Dk / 4;
    const unsigned grid = (unsigned)((quads + 255) / 256);
    if (dtype == QS_BF16) delta_shared_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, quads);
    else delta_shared_kernel<float><<<grid, 256, 0, stream>>>(a, quads);
    return launched();
}
