// dropout.cu -- dropout from a counter-based generator, added on a residual, and its
// gradient.
//
// Mathematics.  Value i is kept where word i % 4 of Philox4x32-10 at the counter
// (i / 4, offset) is at least floor(p 2^32); kept values are divided by 1 - p.  The words
// depend on the key and i alone, so the gradient makes them again and no mask is stored.
// Values are selected, not multiplied: a dropped NaN is gone.
//
// Bound: fp32, memory (8 or 12 bytes a value: 60 us with a residual, 44 us without at 32 M values,
// 0.99 and 0.91 of a copy's rate); bfloat16, arithmetic (the generator's two 32 x 32 -> 64 bit products a
// round for four values keep their pipe busy for 65 and 61% of the time, the other integer pipe 54%, issue
// slots 60 and 56%: 87 and 70 us at 64 M values, 0.68 and 0.56).  CTAs are persistent: a
// thread makes the rounds' keys once, and its next piece is on its way while one is worked on.
#include <cmath>

#include "mixer_device.cuh"
#include "quat_block.h"
#include "quat_host.h"

namespace {

constexpr int kThreads = 256, kCtas = 5, kResCtas = 4;   // CTAs per SM, what their registers allow

struct DropArgs {
    const long long *key;
    const void *x, *res;
    void *y;
    long long n;
    uint32_t least;   // floor(p 2^32) - 1: a word above it is kept (p = 1: none is)
    bool all;         // p = 0
    float scale;
};

struct Philox {
    uint32_t k0[10], k1[10], o1, low, high;   // low, high: the first round's product with the offset
    __device__ __forceinline__ explicit Philox(const long long *key) {
        const unsigned long long seed = (unsigned long long)__ldg(key), offset = (unsigned long long)__ldg(key + 1);
        k0[0] = (uint32_t)seed, k1[0] = (uint32_t)(seed >> 32), o1 = (uint32_t)(offset >> 32);
        const unsigned long long q = (offset & 0xffffffffull) * 0xCD9E8D57u;
        low = (uint32_t)q, high = (uint32_t)(q >> 32);
#pragma unroll
        for (int i = 1; i < 10; ++i) k0[i] = k0[i - 1] + 0x9E3779B9u, k1[i] = k1[i - 1] + 0xBB67AE85u;
    }
    __device__ __forceinline__ uint4 words(unsigned long long block) const {
        const unsigned long long first = (block & 0xffffffffull) * 0xD2511F53u;
        uint32_t c0 = high ^ (uint32_t)(block >> 32) ^ k0[0], c1 = low, c2 = (uint32_t)(first >> 32) ^ o1 ^ k1[0], c3 = (uint32_t)first;
#pragma unroll
        for (int i = 1; i < 10; ++i) {
            const unsigned long long p = (unsigned long long)c0 * 0xD2511F53u, q = (unsigned long long)c2 * 0xCD9E8D57u;
            c0 = (uint32_t)(q >> 32) ^ c1 ^ k0[i], c1 = (uint32_t)q;
            c2 = (uint32_t)(p >> 32) ^ c3 ^ k1[i], c3 = (uint32_t)p;
        }
        return make_uint4(c0, c1, c2, c3);
    }
};

// VEC values at a time: 8 in one access of bfloat16 or two of fp32 (all pointers 16-byte
// aligned; what is left of the last piece one by one), or 4 one by one.
template <typename T, int VEC, bool WIDE, bool RES>
__global__ void __launch_bounds__(kThreads, RES ? kResCtas : kCtas) dropout_kernel(const DropArgs a) {
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    T *y = static_cast<T *>(a.y);
    const long long step = (long long)gridDim.x * kThreads * VEC;
    long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) * VEC;
    struct Piece {
        qs::RawQuads<VEC / 4, T> v;
    } px, pr;
    auto whole = [&](long long at) { return WIDE && at + VEC <= a.n; };
    auto fetch = [&](long long at) {
        if (!whole(at)) return;
        px.v.load(x + at);
        if (RES) pr.v.load(res + at);
    };
    fetch(i);
    const Philox gen(a.key);
    for (; i < a.n; i += step) {
        float4 v[VEC / 4], r[VEC / 4];
        if (whole(i)) {
            px.v.get(v);
            if (RES) pr.v.get(r);
        } else {
            float *f = reinterpret_cast<float *>(v), *g = reinterpret_cast<float *>(r);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                f[k] = i + k < a.n ? qs::load1(x + i + k) : 0.f;
                g[k] = RES && i + k < a.n ? qs::load1(res + i + k) : 0.f;
            }
        }
        fetch(i + step);
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
            const uint4 w = gen.words((unsigned long long)i / 4 + k);
            v[k].x = w.x > a.least || a.all ? v[k].x * a.scale : 0.f;
            v[k].y = w.y > a.least || a.all ? v[k].y * a.scale : 0.f;
            v[k].z = w.z > a.least || a.all ? v[k].z * a.scale : 0.f;
            v[k].w = w.w > a.least || a.all ? v[k].w * a.scale : 0.f;
            if (RES) v[k] = qs::q_add(r[k], v[k]);
        }
        if (whole(i)) {
            qs::store_quads<VEC / 4>(y + i, v);
        } else {
            const float *f = reinterpret_cast<const float *>(v);
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (i + k < a.n) qs::store1(y + i + k, f[k]);
        }
    }
}

template <typename T, int VEC, bool WIDE>
int launch(const DropArgs &a, int sms, cudaStream_t stream) {
    auto go = [&](auto kernel, int ctas) {
        const long long all = (a.n + (long long)VEC * kThreads - 1) / ((long long)VEC * kThreads), most = (long long)sms * ctas;
        kernel<<<(unsigned)(all < most ? all : most), kThreads, 0, stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? QS_OK : QS_ERR_CUDA;
    };
    return a.res ? go(dropout_kernel<T, VEC, WIDE, true>, kResCtas) : go(dropout_kernel<T, VEC, WIDE, false>, kCtas);
}

int run(int dtype, double p, const int64_t *key, const void *x, const void *res, void *y, int64_t n, void *stream_) {
    if ((dtype != QS_F32 && dtype != QS_BF16) || !(p >= 0.0 && p <= 1.0) || n < 0 || n >= int64_t(1) << 40) return QS_ERR_DIMS;
    if (n == 0) return QS_OK;
    if (!x || !y || !key) return QS_ERR_NULL;
    const int es = dtype == QS_BF16 ? 2 : 4;
    const auto skew = [](const void *p, int m) { return reinterpret_cast<uintptr_t>(p) % m != 0; };
    if (skew(x, es) || skew(res, es) || skew(y, es) || skew(key, 8)) return QS_ERR_MISALIGNED;
    const size_t bytes = (size_t)n * es;
    if (qsh::overlaps(y, bytes, x, bytes) || qsh::overlaps(y, bytes, res, bytes) || qsh::overlaps(y, bytes, key, 16)) return QS_ERR_ALIAS;
    int dev = 0, sms = 0;
    const int rc = qsh::device(&dev, &sms);
    if (rc != QS_OK) return rc;
    const uint64_t drop = (uint64_t)std::floor(p * 4294967296.0);
    DropArgs a{};
    a.key = reinterpret_cast<const long long *>(key), a.x = x, a.res = res, a.y = y, a.n = n;
    a.all = drop == 0, a.least = a.all ? 0u : (uint32_t)(drop - 1);
    a.scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
    const bool wide = !qsh::misaligned(x) && !qsh::misaligned(res) && !qsh::misaligned(y);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (dtype == QS_BF16) return wide ? launch<__nv_bfloat16, 8, true>(a, sms, stream) : launch<__nv_bfloat16, 4, false>(a, sms, stream);
    return wide ? launch<float, 8, true>(a, sms, stream) : launch<float, 4, false>(a, sms, stream);
}

}  // namespace

extern "C" int quat_dropout_fwd(int dtype, double p, const int64_t *key, const void *x, const void *residual, void *y,
                                int64_t n, void *stream) {
    return run(dtype, p, key, x, residual, y, n, stream);
}

extern "C" int quat_dropout_bwd(int dtype, double p, const int64_t *key, const void *d_y, void *d_x, int64_t n, void *stream) {
    return run(dtype, p, key, d_y, nullptr, d_x, n, stream);
}
