// delta_rule.cu -- the gated delta rule over whole sequences: forward, and
// backward from the forward's carries and errors.  The kernels are in
// delta_fwd_tc.cuh (forward walk), delta_chain_tc.cuh (backward: the chain of the
// states' cotangents) and delta_bwd_tc.cuh (backward: the gradients of each chunk).
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

// Joins the segments of a sequence: from the state that enters the first (backward: the
// cotangent that leaves the last), the state that enters each, m' = map m + own.  A CTA
// takes 16 value columns of one (sequence, head); two threads a row of dk.  Bound: the chain
// of segments, each a round of loads of the map (2.3 us a segment; 1 x 16384 x 16 x 64 in 9
// segments 20.6 us, 4 x 1000 x 8 x 64 in 4 segments 9.2 us).
template <bool BWD>
__global__ void __launch_bounds__(256) delta_join_kernel(const DeltaArgs a, const float *first, float *out) {
    __shared__ float m[QS_DELTA_MAX_D][20];
    const int r = threadIdx.x / 2, c = threadIdx.x % 2 * 8, x0 = blockIdx.y * 16 + c;
    const bool in = r < a.Dk && x0 < a.Dv;
    const size_t nh = blockIdx.x, elem = (size_t)r * a.Dv + x0;
    store4(&m[r][c], q_zero()), store4(&m[r][c + 4], q_zero());   // (rows past Dk stay zero)
    float4 v[2] = {q_zero(), q_zero()};
    if (first && in) {
        const float4 *p = reinterpret_cast<const float4 *>(first + nh * a.Dk * a.Dv + elem);
        v[0] = __ldg(p), v[1] = __ldg(p + 1);
    }
    for (int i = 0; i < a.segs; ++i) {
        const size_t at = nh * a.segs + (BWD ? a.segs - 1 - i : i);
        if (in) {
            float *p = out + at * a.Dk * a.Dv + elem;
            store4(p, v[0]), store4(p + 4, v[1]);
        }
        if (i + 1 == a.segs) break;
        __syncthreads();
        if (r < a.Dk) store4(&m[r][c], v[0]), store4(&m[r][c + 4], v[1]);
        __syncthreads();
        v[0] = v[1] = q_zero();
        if (in) {
            const float4 *p = reinterpret_cast<const float4 *>(a.seg_own + at * a.Dk * a.Dv + elem);
            v[0] = __ldg(p), v[1] = __ldg(p + 1);
            const float4 *f = reinterpret_cast<const float4 *>(a.seg_map + (at * a.Dk + r) * a.Dk);
            for (int j0 = 0; j0 < a.Dk; j0 += 32) {   // eight loads of the map's row at a time (its columns past Dk count as zero)
                float4 w8[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) w8[k] = j0 + 4 * k < a.Dk ? __ldg(f + j0 / 4 + k) : q_zero();
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    const float w[4] = {w8[k / 4].x, w8[k / 4].y, w8[k / 4].z, w8[k / 4].w};
                    const float4 x = *reinterpret_cast<const float4 *>(&m[j0 + k][c]), y = *reinterpret_cast<const float4 *>(&m[j0 + k][c + 4]);
                    const float f1 = w[k % 4];
                    v[0] = make_float4(fmaf(f1, x.x, v[0].x), fmaf(f1, x.y, v[0].y), fmaf(f1, x.z, v[0].z), fmaf(f1, x.w, v[0].w));
                    v[1] = make_float4(fmaf(f1, y.x, v[1].x), fmaf(f1, y.y, v[1].y), fmaf(f1, y.z, v[1].z), fmaf(f1, y.w, v[1].w));
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
int launched() { return cudaGetLastError() == cudaSuccess ? QS_OK : QS_ERR_CUDA; }

// Cuts each sequence into segments where there are too few (sequence, head) pairs to fill
// the GPU: a first walk sums every segment but one up as an affine map of its state, the
// join runs over the segments, and the real walk starts each from its own state.  The
// rule is the cost in chunk steps: waves of CTAs times chunks per segment, a summing
// walk counted as 0.9 of a real one (139 and 151 us on 1 x 16384 x 16 x 64), a join step as
// 0.4 of a chunk, the two launches as 3.  (1 x 131072 x 16 x 64: 19 segments, 2.1 instead of
// 9.8 ms; 1 x 4096 x 48 x 128 whole 363 us, in three segments 419; 8 x 4096 x 16 x 128 has
// enough pairs: one.)
//
// Packed sequences, whose lengths only the device knows, are walked whole, the longest
// first where they do not all run at once: a long one that starts last is the call's tail
// (mean of six draws of lengths, heads of 128, in order and sorted: 17 sequences of 4333
// steps 122 and 108 us, 64 of 32768 481 and 392, 100 of 65536 838 and 734, 128 of 17000 334
// and 329).  Sorting costs each CTA about 1 us, which many sequences of under 128 steps,
// even by themselves, do not win back.
void cut(DeltaArgs &a, int sms) {
    a.segs = 1, a.seg_chunks = a.NC, a.sms = sms;
    a.longest_first = a.offsets && a.N > 1 && a.N <= kMostOrdered && a.N * a.Hv > sms && a.S >= 128 * a.N;
    if (a.offsets || a.NC < 4) return;
    const long long pairs = a.N * a.Hv, kinds = a.Dk <= 64 && a.Dv <= 64 ? 1 : 2;
    double best = (double)a.NC * ((pairs + sms - 1) / sms) * 0.9;   // cut only for a clear gain
    for (long long want = 2; want <= 64 && want <= a.NC && pairs * want <= 2 * sms; ++want) {
        const long long sc = (a.NC + want - 1) / want, n = (a.NC + sc - 1) / sc;
        if (n < 2) continue;
        const double waves = (double)((pairs * n + sms - 1) / sms) + 0.9 * (double)((pairs * kinds * (n - 1) + sms - 1) / sms);
        const double cost = waves * sc + 0.4 * n + 3;
        if (cost < best) best = cost, a.segs = (int)n, a.seg_chunks = sc;
    }
}

size_t seg_floats(const DeltaArgs &a) {   // of seg_m, seg_own and seg_map, one after the other
    return a.segs > 1 ? (size_t)(a.N * a.Hv) * a.segs * ((size_t)a.Dk * a.Dv * 2 + (size_t)a.Dk * a.Dk) : 0;
}

// A walk over the chunks, one CTA per (sequence, value head) or segment of one.
template <bool BWD, typename T, int NT>
int launch_walks(DeltaArgs &a, float *seg, cudaStream_t stream) {
    constexpr int PT = BWD || NT == 3 ? 3 : 2;
    CUtensorMap maps[3];
    if (NT == 1 && a.B * a.S > 0) {
        const qsh::Strides so = {(long long)(a.S * a.Hv * a.Dv), (long long)a.Hv * a.Dv, a.Dv};
        int rc = qsh::head_map(&maps[0], a.k, a.sk, a.B, a.S, a.Hk, a.Dk);
        if (rc == QS_OK) rc = qsh::head_map(&maps[1], a.q, a.sq, a.B, a.S, a.Hk, a.Dk);
        if (rc == QS_OK) rc = BWD ? qsh::head_map(&maps[2], a.d_o, so, a.B, a.S, a.Hv, a.Dv)
                                  : qsh::head_map(&maps[2], a.v, a.sv, a.B, a.S, a.Hv, a.Dv);
        if (rc != QS_OK) return rc;
    }
    auto go = [&](auto kernel, size_t smem, long long grid) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
            cudaGetLastError();
            return (int)QS_ERR_CUDA;
        }
        kernel<<<(unsigned)grid, kWalkThreads, smem, stream>>>(a, maps[0], maps[1], maps[2]);
        return launched();
    };
    auto walk = [&](auto sum, long long grid) {
        constexpr bool SUM = decltype(sum)::value;
        constexpr size_t small = WalkLayout<NT, 64, PT>::BYTES, large = WalkLayout<NT, 128, PT>::BYTES;
        if constexpr (BWD)
            return a.Dk <= 64 ? go(delta_chain_tc_kernel<T, NT, 64, SUM>, small, grid)
                              : go(delta_chain_tc_kernel<T, NT, 128, SUM>, large, grid);
        else
            return a.Dk <= 64 ? go(delta_fwd_tc_kernel<T, NT, 64, SUM>, small, grid)
                              : go(delta_fwd_tc_kernel<T, NT, 128, SUM>, large, grid);
    };
    const long long pairs = a.N * a.Hv;
    if (a.segs > 1) {
        const size_t states = (size_t)pairs * a.segs * a.Dk * a.Dv;
        a.seg_m = seg, a.seg_own = seg + states, a.seg_map = seg + 2 * states;
        int rc = walk(std::true_type(), pairs * (a.segs - 1) * (a.Dk <= 64 && a.Dv <= 64 ? 1 : 2));
        if (rc != QS_OK) return rc;
        delta_join_kernel<BWD><<<dim3((unsigned)pairs, (unsigned)(a.Dv + 15) / 16), 256, 0, stream>>>(a, BWD ? a.d_final : a.init, seg);
        rc = launched();
        if (rc != QS_OK) return rc;
    }
    return walk(std::false_type(), pairs * a.segs);
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
    const int64_t heads = Hv > Hk ? Hv : Hk;
    if ((__int128)N * Hv >= lim || (__int128)slots * Hv >= lim || (__int128)B * S * heads >= ((__int128)1 << 40)) return QS_ERR_DIMS;
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

// Strides that the kernels cannot take.  (bfloat16 rows come by tensor maps, fp32 rows by plain loads.)
bool bad_layout(const DeltaArgs &a, int dtype) {
    const int es = dtype == QS_BF16 ? 2 : 4;
    if (qsh::bad_strides(a.sq, es) || qsh::bad_strides(a.sk, es) || qsh::bad_strides(a.sv, es)) return true;
    return dtype == QS_BF16 && (qsh::has_flat_dim(a.sq, a.B, a.S, a.Hk) || qsh::has_flat_dim(a.sk, a.B, a.S, a.Hk) ||
                                qsh::has_flat_dim(a.sv, a.B, a.S, a.Hv));
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
    if (strides && bad_layout(a, dtype)) return QS_ERR_MISALIGNED;
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
    cut(a, sms);
    qsh::Hold hold;
    const int wc = qsh::workspace(dev, stream, sizeof(WsHeader) + seg_floats(a) * 4, &ws, &hold);
    if (wc != QS_OK) return wc;
    float *seg = reinterpret_cast<float *>(ws + sizeof(WsHeader));
    a.ctl = {reinterpret_cast<WsHeader *>(ws), qsh::stall_tile(), qsh::timeout_ns()};
    return dtype == QS_BF16 ? launch_walks<false, __nv_bfloat16, 1>(a, seg, stream) : launch_walks<false, float, 3>(a, seg, stream);
}

extern "C" int quat_delta_bwd(int dtype, int gate_dtype, float scale, const void *q, const void *k, const void *v,
                              const void *g, const void *beta, const float *carries, const float *errors, const void *d_o,
                              const float *d_final, void *d_q, void *d_k, void *d_v, void *d_g, void *d_beta, float *d_init,
                              const int64_t *strides, const int32_t *offsets, int64_t N, int64_t B, int64_t S, int64_t Hk,
                              int64_t Hv, int64_t Dk, int64_t Dv, void *stream_) {
    const int dc = check(dtype, gate_dtype, offsets, N, B, S, Hk, Hv, Dk, Dv);
    if (dc == 1) {   // keys that no value head uses have zero gradients
        const size_t bytes = (size_t)B * S * Hk * Dk * (dtype == QS_BF16 ? 2 : 4);
        for (void *p : {d_q, d_k}) {
            if (bytes == 0) break;
            if (!p) return QS_ERR_NULL;
            if (cudaMemsetAsync(p, 0, bytes, static_cast<cudaStream_t>(stream_)) != cudaSuccess) {
                cudaGetLastError();
                return QS_ERR_CUDA;
            }
        }
        return QS_OK;
    }
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
    if (strides && bad_layout(a, dtype)) return QS_ERR_MISALIGNED;
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
    cut(a, sms);
    qsh::Hold hold;
    rc = qsh::workspace(dev, stream, sizeof(WsHeader) + nds + nw + 2 * nh + seg_floats(a) * 4, &ws, &hold);
    if (rc != QS_OK) return rc;
    a.q = q, a.k = k, a.v = v, a.g = g, a.beta = beta, a.carries_in = carries, a.errors_in = errors, a.d_o = d_o;
    a.d_final = d_final, a.dq = d_q, a.dk = d_k, a.dv = d_v, a.dg = d_g, a.dbeta = d_beta, a.d_init = d_init;
    unsigned char *p = ws + sizeof(WsHeader);
    a.ds = reinterpret_cast<float *>(p), a.w = reinterpret_cast<float *>(p + nds);
    a.dqh = reinterpret_cast<float *>(p + nds + nw), a.dkh = reinterpret_cast<float *>(p + nds + nw + nh);
    a.ctl = {reinterpret_cast<WsHeader *>(ws), qsh::stall_tile(), qsh::timeout_ns()};
    float *seg = reinterpret_cast<float *>(p + nds + nw + 2 * nh);
    rc = dtype == QS_BF16 ? launch_walks<true, __nv_bfloat16, 1>(a, seg, stream) : launch_walks<true, float, 3>(a, seg, stream);
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
