// dropout.cu -- dropout from a counter-based generator, added on a residual, and its
// gradient.
//
// Mathematics.  Value i is kept where word i % 4 of Philox4x32-10 at the counter
// (i / 4, offset) is at least floor(p 2^32); kept values are divided by 1 - p.  The words
// depend on the key and i alone, so the gradient makes them again and no mask is stored.
// Values are selected, not multiplied: a dropped NaN is gone.
//
// Bound: memory (4 to 6 bytes a value in bfloat16) against about 15 instructions a value
// (two 32 x 32 -> 64 bit products a round for four values).
#include <cmath>

#include "mixer_device.cuh"
#include "quat_block.h"
#include "quat_host.h"

namespace {

constexpr int kThreads = 256, kPer = 2;   // pieces of VEC values per thread

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
    uint32_t k0, k1, o0, o1;
    __device__ __forceinline__ explicit Philox(const long long *key) {
        const unsigned long long seed = (unsigned long long)__ldg(key), offset = (unsigned long long)__ldg(key + 1);
        k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32), o0 = (uint32_t)offset, o1 = (uint32_t)(offset >> 32);
    }
    __device__ __forceinline__ uint4 words(unsigned long long block) const {
        uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = o0, c3 = o1, a = k0, b = k1;
#pragma unroll
        for (int i = 0; i < 10; ++i) {
            const unsigned long long p = (unsigned long long)c0 * 0xD2511F53u, q = (unsigned long long)c2 * 0xCD9E8D57u;
            c0 = (uint32_t)(q >> 32) ^ c1 ^ a, c1 = (uint32_t)q;
            c2 = (uint32_t)(p >> 32) ^ c3 ^ b, c3 = (uint32_t)p;
            a += 0x9E3779B9u, b += 0xBB67AE85u;
        }
        return make_uint4(c0, c1, c2, c3);
    }
};

// VEC values at a time: 8 of bfloat16 or 4 of fp32 in one access (all pointers 16-byte
// aligned), or 4 one by one.
template <typename T, int VEC, bool WIDE>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropArgs a) {
    const T *x = static_cast<const T *>(a.x), *res = static_cast<const T *>(a.res);
    T *y = static_cast<T *>(a.y);
    const Philox gen(a.key);
    const long long first = ((long long)blockIdx.x * kPer * kThreads + threadIdx.x) * VEC;
    float4 v[kPer][VEC / 4], r[kPer][VEC / 4];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const long long i = first + (long long)j * kThreads * VEC;
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) v[j][k] = r[j][k] = qs::q_zero();
        if (WIDE && i + VEC <= a.n) {
            qs::load_quads<VEC / 4>(x + i, v[j]);
            if (res) qs::load_quads<VEC / 4>(res + i, r[j]);
        } else if (i < a.n) {
            float *f = reinterpret_cast<float *>(v[j]), *g = reinterpret_cast<float *>(r[j]);
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (i + k < a.n) {
                    f[k] = qs::load1(x + i + k);
                    if (res) g[k] = qs::load1(res + i + k);
                }
        }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const long long i = first + (long long)j * kThreads * VEC;
        if (i >= a.n) return;
#pragma unroll
        for (int k = 0; k < VEC / 4; ++k) {
            const uint4 w = gen.words((unsigned long long)i / 4 + k);
            v[j][k].x = r[j][k].x + (w.x > a.least || a.all ? v[j][k].x * a.scale : 0.f);
            v[j][k].y = r[j][k].y + (w.y > a.least || a.all ? v[j][k].y * a.scale : 0.f);
            v[j][k].z = r[j][k].z + (w.z > a.least || a.all ? v[j][k].z * a.scale : 0.f);
            v[j][k].w = r[j][k].w + (w.w > a.least || a.all ? v[j][k].w * a.scale : 0.f);
        }
        if (WIDE && i + VEC <= a.n) {
            qs::store_quads<VEC / 4>(y + i, v[j]);
        } else {
            const float *f = reinterpret_cast<const float *>(v[j]);
#pragma unroll
            for (int k = 0; k < VEC; ++k)
                if (i + k < a.n) qs::store1(y + i + k, f[k]);
        }
    }
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
    const int vec = wide && dtype == QS_BF16 ? 8 : 4;
    const unsigned grid = (unsigned)((n + (int64_t)vec * kPer * kThreads - 1) / ((int64_t)vec * kPer * kThreads));
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (dtype == QS_BF16) {
        if (wide) dropout_kernel<__nv_bfloat16, 8, true><<<grid, kThreads, 0, stream>>>(a);
        else dropout_kernel<__nv_bfloat16, 4, false><<<grid, kThreads, 0, stream>>>(a);
    } else {
        if (wide) dropout_kernel<float, 4, true><<<grid, kThreads, 0, stream>>>(a);
        else dropout_kernel<float, 4, false><<<grid, kThreads, 0, stream>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? QS_OK : QS_ERR_CUDA;
}

}  // namespace

extern "C" int quat_dropout_fwd(int dtype, double p, const int64_t *key, const void *x, const void *residual, void *y,
                                int64_t n, void *stream) {
    return run(dtype, p, key, x, residual, y, n, stream);
}

extern "C" int quat_dropout_bwd(int dtype, double p, const int64_t *key, const void *d_y, void *d_x, int64_t n, void *stream) {
    return run(dtype, p, key, d_y, nullptr, d_x, n, stream);
}
