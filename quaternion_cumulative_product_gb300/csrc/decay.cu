// decay.cu -- linear attention with a decay for each head over whole sequences: forward and
// backward.
//
// bfloat16: the walk of decay_walk.cuh; backward three of them (dq, dk, dv) and decay_gate.cuh.
// fp32, whose values are three terms each and take three times the room: the states of all chunks
// at once (decay_states.cuh), then the delta rule's kernels without its errors (RULE,
// delta_prep.cuh).  4 x 1000 x 8 heads of 64, fp32, both ways: 194 us; with the states walked,
// twice where sequences are cut, 326 us.
#include <algorithm>

#include "decay_gate.cuh"
#include "decay_states.cuh"
#include "delta_host.cuh"

using namespace qs;

namespace {

int early(cudaError_t e) {
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? QS_OK : QS_ERR_CUDA;
}

// fp32: cuts sequences into as many segments as fill the GPU (their states come from all chunks at once).
//
// Packed sequences, whose lengths only the device knows, are cut into an SM's share of all chunks, and at least 8,
// where they are longer by half (a chunk takes 6 us of a walk at heads of 64 and 12 at 128, the states two
// launches more): a batch of like sequences that fills the GPU is walked whole, and its states are not made.
// Forward, 2 sequences of 65536 steps in all, a head of 128: 327 us (whole 5970 to 11630); 10 of 16889, 8
// heads of 128 and 64: 389 (1120); 20 of 4305, 8 heads of 32 and 80, none of them cut: 119 (104).
void cut_states(DeltaArgs &a, int sms) {
    a.segs = 1, a.seg_chunks = a.NC, a.sms = sms;
    a.longest_first = a.offsets && a.N > 1 && a.N <= kMostOrdered && a.N * a.Hv > sms && a.S >= 128 * a.N;
    if (a.offsets) {
        const long long share = std::max<long long>((a.slots * a.Hv + sms - 1) / sms, 8);
        if (a.NC >= 2 * share) a.seg_chunks = share, a.uncut = share + share / 2;
        return;
    }
    const long long pairs = a.N * a.Hv, want = pairs ? sms / pairs : 0;
    if (want < 2 || a.NC < 2) return;
    a.seg_chunks = (a.NC + want - 1) / want, a.segs = (int)((a.NC + a.seg_chunks - 1) / a.seg_chunks);
}

int launch_states(const StateArgs &s, unsigned sides, cudaStream_t stream) {
    const DeltaArgs &d = s.d;
    auto own = [&](auto kernel, int D) {
        const int smem = 2 * DC * D * 4;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
            cudaGetLastError();
            return (int)QS_ERR_CUDA;
        }
        kernel<<<dim3((unsigned)(d.slots * d.Hv), sides), kOwnThreads, smem, stream>>>(s);
        return launched();
    };
    if (d.slots > 0) {
        const int rc = d.Dk <= 64 && d.Dv <= 64 ? own(decay_own_kernel<64>, 64) : own(decay_own_kernel<128>, 128);
        if (rc != QS_OK) return rc;
    }
    const long long parts = (d.Dk * d.Dv / 4 + 255) / 256;
    if (d.N * d.Hv * parts >= 1ll << 31) return QS_ERR_DIMS;
    const dim3 grid((unsigned)(d.N * d.Hv * parts), sides);
    if (d.slots > 0) return early(qsh::launch_next(decay_run_kernel, grid, 256, 0, stream, s, (unsigned)parts));
    decay_run_kernel<<<grid, 256, 0, stream>>>(s, (unsigned)parts);   // the call's first kernel: it reads what others have left on the stream
    return launched();
}

// Cuts each sequence into segments where there are too few walks to fill the GPU: a first walk
// sums up every segment but one, the join hands the states on, and the real walk starts each
// segment from its own.  Costs are in chunks; a summing walk counts as half a real one (1 x 131072 x
// 16 x 64: 125 and 277 us).
void cut_walks(DecayArgs &a, int sms) {
    a.segs = 1, a.seg_chunks = a.NC;
    a.longest_first = a.offsets && a.N > 1 && a.N <= kMostOrdered && a.N * a.Hv > sms && a.S >= 128 * a.N;
    if (a.offsets || a.NC < 4) return;
    const long long pairs = a.N * a.Hv;
    double best = (double)a.NC * ((pairs + sms - 1) / sms) * 0.9;   // cut only for a clear gain
    for (long long want = 2; want <= 64 && want <= a.NC && pairs * want <= 4 * sms; ++want) {
        const long long sc = (a.NC + want - 1) / want, n = (a.NC + sc - 1) / sc;
        if (n < 2) continue;
        const double waves = (double)((pairs * n + sms - 1) / sms) + 0.5 * (double)((pairs * (n - 1) + sms - 1) / sms);
        const double cost = waves * sc + 0.1 * n + 3;
        if (cost < best) best = cost, a.segs = (int)n, a.seg_chunks = sc;
    }
}

size_t walk_floats(const DecayArgs &a, int D) {   // of seg_m, seg_own and seg_decay
    return a.segs > 1 ? (size_t)(a.N * a.Hv) * a.segs * (2 * (size_t)D * D + 4) : 0;
}

// A walk of KIND, in segments with their sums and the join before it.
// `next`: not the call's first launch.
template <int D, WalkKind KIND>
int launch_decay(DecayArgs &a, float *seg, bool next, cudaStream_t stream) {
    constexpr bool REV = KIND == WALK_DK || KIND == WALK_DV;
    auto go = [&](auto kernel, size_t smem, long long grid) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
            cudaGetLastError();
            return (int)QS_ERR_CUDA;
        }
        if (next) return early(qsh::launch_next(kernel, (unsigned)grid, kDecayThreads, smem, stream, a));
        kernel<<<(unsigned)grid, kDecayThreads, smem, stream>>>(a);
        return launched();
    };
    const long long pairs = a.N * a.Hv;
    if (a.segs > 1) {
        const size_t n = (size_t)pairs * a.segs;
        DecayRole &r = a.role;
        r.seg_m = seg, r.seg_own = seg + n * D * D, r.seg_decay = seg + 2 * n * D * D;
        if constexpr (KIND != WALK_DV) {   // (which takes the states of dk, just walked: the same, transposed)
            int rc = go(decay_walk_kernel<D, REV ? WALK_SUM_REV : WALK_SUM>, DecayLayout<D, true, false>::BYTES, pairs * (a.segs - 1));
            if (rc != QS_OK) return rc;
            rc = early(qsh::launch_next(decay_join_kernel<D, REV>, dim3(D * D / 1024, (unsigned)pairs), 256, 0, stream, a));
            if (rc != QS_OK) return rc;
            next = true;
        }
    }
    return go(decay_walk_kernel<D, KIND>, DecayLayout<D, false, KIND == WALK_DQ || KIND == WALK_DK>::BYTES, pairs * a.segs);
}
template <WalkKind KIND>
int launch_walk(DecayArgs &a, int D, float *seg, bool next, cudaStream_t stream) {
    return D == 64 ? launch_decay<64, KIND>(a, seg, next, stream) : launch_decay<128, KIND>(a, seg, next, stream);
}

// A tensor [B, S, H, D] that a walk reads.
struct Rows {
    const void *p;
    qsh::Strides st;
    int64_t H, D;
};

int set_role(DecayRole &r, const DecayArgs &a, const Rows &x, const Rows &y, const Rows &z) {
    r.gx = (int)(a.Hv / x.H), r.gy = (int)(a.Hv / y.H), r.gz = (int)(a.Hv / z.H);
    r.dk = (int)x.D, r.dv = (int)z.D;
    if (a.B * a.S == 0) return QS_OK;
    int rc = qsh::head_map(&r.x, x.p, x.st, a.B, a.S, x.H, x.D);
    if (rc == QS_OK) rc = qsh::head_map(&r.y, y.p, y.st, a.B, a.S, y.H, y.D);
    if (rc == QS_OK) rc = qsh::head_map(&r.z, z.p, z.st, a.B, a.S, z.H, z.D);
    return rc;
}

void set_walks(DecayArgs &a, const DeltaArgs &d) {
    a.g = d.g, a.offsets = d.offsets, a.B = d.B, a.S = d.S, a.N = d.N, a.NC = (d.S + WC - 1) / WC, a.Hv = d.Hv;
    a.gate16 = d.gate16, a.scale = d.scale;
}

// `out` [B, S, Hv, dv] of a role, bfloat16 (by TMA) or fp32.
int set_out(DecayRole &r, const DecayArgs &a, void *out, int64_t dv, bool fp32) {
    r.out = out, r.out32 = fp32;
    if (fp32 || a.B * a.S == 0) return QS_OK;
    return qsh::head_map(&r.o, out, {(long long)(a.S * a.Hv * dv), (long long)a.Hv * dv, (long long)dv}, a.B, a.S, a.Hv, dv);
}

int forward16(const DeltaArgs &d, int dev, int sms, cudaStream_t stream) {
    DecayArgs a{};
    set_walks(a, d);
    DecayRole &r = a.role;
    int rc = set_role(r, a, {d.q, d.sq, d.Hk, d.Dk}, {d.k, d.sk, d.Hk, d.Dk}, {d.v, d.sv, d.Hv, d.Dv});
    if (rc == QS_OK) rc = set_out(r, a, d.o, d.Dv, false);
    if (rc != QS_OK) return rc;
    r.init = d.init, r.fin = d.fin, r.lane = 1, r.col = d.Dv;
    cut_walks(a, sms);
    const int D = d.Dk <= 64 && d.Dv <= 64 ? 64 : 128;
    unsigned char *ws = nullptr;
    qsh::Hold hold;
    rc = qsh::workspace(dev, stream, sizeof(WsHeader) + walk_floats(a, D) * 4, &ws, &hold);
    if (rc != QS_OK) return rc;
    a.ctl = {reinterpret_cast<WsHeader *>(ws), qsh::stall_tile(), qsh::timeout_ns()};
    float *seg = reinterpret_cast<float *>(ws + sizeof(WsHeader));
    return launch_walk<WALK_OUT>(a, D, seg, false, stream);
}

template <int D>
int launch_gates(const GateArgs &a, int sms, cudaStream_t stream) {
    constexpr int smem = GateLayout<D>::BYTES;
    if (cudaFuncSetAttribute(decay_gate_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
        cudaGetLastError();
        return QS_ERR_CUDA;
    }
    return early(qsh::launch_next(decay_gate_kernel<D>, (unsigned)std::min<long long>(a.slots * a.Hv, 2 * sms), kGateThreads, smem, stream, a));
}

// dq and (with the states that it leaves) dk and dv are walks, dg a kernel of its own.
int backward16(const DeltaArgs &d, int dev, int sms, cudaStream_t stream) {
    DecayArgs a{};
    set_walks(a, d);
    cut_walks(a, sms);
    const qsh::Strides so = {(long long)(d.S * d.Hv * d.Dv), (long long)d.Hv * d.Dv, d.Dv};
    const Rows q = {d.q, d.sq, d.Hk, d.Dk}, k = {d.k, d.sk, d.Hk, d.Dk}, v = {d.v, d.sv, d.Hv, d.Dv}, o = {d.d_o, so, d.Hv, d.Dv};
    const int D = d.Dk <= 64 && d.Dv <= 64 ? 64 : 128, group = d.Hv / d.Hk;
    const bool shared = d.Hv != d.Hk;
    const long long slots = d.offsets ? d.S / WC + d.N : d.N * a.NC;
    const size_t rows = (size_t)d.B * d.S * d.Hv, nstate = align256((size_t)slots * d.Hv * D * D * 4), ndots = align256(2 * rows * 4),
                 ncross = align256((size_t)slots * d.Hv * 8 * 4), nh = shared ? align256(rows * d.Dk * 4) : 0;
    unsigned char *ws = nullptr;
    qsh::Hold hold;
    int rc = qsh::workspace(dev, stream, sizeof(WsHeader) + nstate + 2 * ndots + ncross + 2 * nh + walk_floats(a, D) * 4, &ws, &hold);
    if (rc != QS_OK) return rc;
    unsigned char *p = ws + sizeof(WsHeader);
    auto part = [&](size_t n) {
        float *at = reinterpret_cast<float *>(p);
        p += n;
        return at;
    };
    float *states = part(nstate), *dota = part(ndots), *dotb = part(ndots), *cross = part(ncross), *dqh = part(nh), *dkh = part(nh), *seg = part(0);
    a.ctl = {reinterpret_cast<WsHeader *>(ws), qsh::stall_tile(), qsh::timeout_ns()};
    GateArgs g{};
    DecayRole &r = a.role;
    rc = set_role(r, a, o, v, k);
    if (rc == QS_OK) rc = set_out(r, a, shared ? dqh : d.dq, d.Dk, shared);
    if (rc != QS_OK) return rc;
    if (d.B * d.S > 0) rc = qsh::head_map(&r.b, d.q, d.sq, d.B, d.S, d.Hk, d.Dk);
    if (rc != QS_OK) return rc;
    r.gb = group, r.dots = dota, r.init = d.init, r.dump = states, r.lane = d.Dv, r.col = 1;
    g.o = r.x, g.v = r.y, g.k = r.z;
    rc = launch_walk<WALK_DQ>(a, D, seg, false, stream);
    r = DecayRole{};
    if (rc == QS_OK) rc = set_role(r, a, v, o, q);
    if (rc == QS_OK) rc = set_out(r, a, shared ? dkh : d.dk, d.Dk, shared);
    if (rc != QS_OK) return rc;
    if (d.B * d.S > 0) rc = qsh::head_map(&r.b, d.k, d.sk, d.B, d.S, d.Hk, d.Dk);
    if (rc != QS_OK) return rc;
    r.gb = group, r.dots = dotb, r.init = d.d_final, r.other = states, r.cross = cross, r.lane = d.Dv, r.col = 1;
    g.q = r.z;
    rc = launch_walk<WALK_DK>(a, D, seg, true, stream);
    r = DecayRole{};
    if (rc == QS_OK) rc = set_role(r, a, k, q, o);
    if (rc == QS_OK) rc = set_out(r, a, d.dv, d.Dv, false);
    if (rc != QS_OK) return rc;
    r.init = d.d_final, r.fin = d.d_init, r.lane = 1, r.col = d.Dv;
    rc = launch_walk<WALK_DV>(a, D, seg, true, stream);
    if (rc != QS_OK || d.B * d.S == 0) return rc;
    g.g = d.g, g.dg = d.dg, g.a = dota, g.b = dotb, g.cross = cross, g.offsets = d.offsets;
    g.B = d.B, g.S = d.S, g.N = d.N, g.NC = a.NC, g.slots = slots, g.Hv = d.Hv, g.shared = group, g.gate16 = d.gate16, g.scale = d.scale, g.ctl = a.ctl;
    rc = D == 64 ? launch_gates<64>(g, sms, stream) : launch_gates<128>(g, sms, stream);
    if (rc != QS_OK || !shared) return rc;
    DeltaArgs sum = d;
    sum.dqh = dqh, sum.dkh = dkh;
    const long long quads = d.B * d.S * d.Hk * d.Dk / 4;
    return early(qsh::launch_next(delta_shared_kernel<__nv_bfloat16>, (unsigned)((quads + 255) / 256), 256, 0, stream, sum, quads));
}

}  // namespace

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
    if (dtype == QS_BF16) return forward16(a, dev, sms, stream);
    unsigned char *ws = nullptr;
    cut_states(a, sms);
    bool parts = a.segs > 1 || a.uncut;
    const size_t kept = parts ? (size_t)a.slots * Hv * Dk * Dv : 0, wholes = parts ? (size_t)a.slots * Hv : 0;
    qsh::Hold hold;
    int wc = qsh::workspace(dev, stream, sizeof(WsHeader) + (kept + wholes) * 4, &ws, &hold);
    if (wc == QS_ERR_NOMEM && a.uncut) {   // no room for the states (half of the tensors' bytes): whole walks, which take none
        hold = {}, parts = false, a.uncut = 0;
        wc = qsh::workspace(dev, stream, sizeof(WsHeader), &ws, &hold);
    }
    if (wc != QS_OK) return wc;
    float *carries = reinterpret_cast<float *>(ws + sizeof(WsHeader));
    a.ctl = {reinterpret_cast<WsHeader *>(ws), qsh::stall_tile(), qsh::timeout_ns()};
    if (parts) wc = launch_states({a, carries + kept, {{carries, init, nullptr, false}}, a.uncut > 0}, 1, stream);
    if (wc != QS_OK) return wc;
    a.carries_in = carries;
    return launch_walks<false, float, 3, false>(a, nullptr, stream);
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
    a.q = q, a.k = k, a.v = v, a.g = g, a.init = init, a.d_o = d_o, a.d_final = d_final;
    a.dq = d_q, a.dk = d_k, a.dv = d_v, a.dg = d_g, a.d_init = d_init;
    if (dtype == QS_BF16) return backward16(a, dev, sms, stream);
    const bool shared = Hv != Hk;
    const size_t nds = align256(kept * 4), nh = shared ? align256((size_t)B * S * Hv * Dk * 4) : 0, nwhole = align256((size_t)a.slots * Hv * 4);
    unsigned char *ws = nullptr;
    cut_states(a, sms);
    qsh::Hold hold;
    rc = qsh::workspace(dev, stream, sizeof(WsHeader) + 2 * nds + 2 * nh + nwhole, &ws, &hold);
    if (rc != QS_OK) return rc;
    unsigned char *p = ws + sizeof(WsHeader);
    float *carries = reinterpret_cast<float *>(p), *whole = reinterpret_cast<float *>(p + 2 * nds + 2 * nh);
    a.ds = reinterpret_cast<float *>(p + nds);
    a.dqh = reinterpret_cast<float *>(p + 2 * nds), a.dkh = reinterpret_cast<float *>(p + 2 * nds + nh);
    a.ctl = {reinterpret_cast<WsHeader *>(ws), qsh::stall_tile(), qsh::timeout_ns()};
    rc = launch_states({a, whole, {{carries, init, nullptr, false}, {a.ds, d_final, d_init, true}}}, 2, stream);   // (without steps: d_init is d_final, or zeros)
    if (rc != QS_OK || !some) return rc;
    a.carries_in = carries, a.d_init = nullptr;
    rc = launch_walks<true, float, 3, false>(a, nullptr, stream);   // dv
    if (rc == QS_OK) rc = launch_chunks<float, 3, 3, false>(a, stream);
    if (rc != QS_OK || !shared) return rc;
    const long long quads = B * S * Hk * Dk / 4;
    delta_shared_kernel<float><<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(a, quads);
    return launched();
}
