// layer_norm.cu -- layer norm over a row and its backward, with the sums of the
// weights' gradients.
//
// Mathematics.  m = mean(x), r = (mean((x - m)^2) + eps)^(-1/2), n = (x - m) r,
// y = n w + b.  With dn = dy w:
//     dx = r (dn - mean(dn) - n mean(dn n)),    dw = sum over rows of dy n,    db = of dy.
// A row stays in registers, so the squares are summed about the mean (x^2 summed up
// would cancel where the mean is far from zero), and dn n as r dn (x - m) in the same round.
//
// Bound: memory.  Every input is read once and every output written once; a row is held
// by 32 .. 1024 threads (a power of two), 16 bytes to an access where rows and pointers
// are aligned so, single values (neighbouring lanes neighbouring values) where not.
#include "mixer_device.cuh"
#include "quat_common.cuh"
#include "quat_block.h"
#include "quat_host.h"

namespace {

struct NormArgs {
    const void *x, *dy;
    const float *w, *b;
    void *y;       // y; backward: d_x
    float *part;   // backward: sums of each CTA [grid][2][D]
    long long R, ld;
    int D;
    float eps, inv_d;
};

// VEC values as they are in memory.
template <typename T, int VEC>
struct Raw;
template <>
struct Raw<float, 4> {
    float4 r;
    __device__ __forceinline__ void load(const float *p) { r = __ldg(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void get(float *f) const { f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w; }
};
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(float *f) const {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
};
template <typename T>
struct Raw<T, 1> {
    T r;
    __device__ __forceinline__ void load(const T *p) { r = *p; }
    __device__ __forceinline__ void get(float *f) const { f[0] = qs::to_float(r); }
};

template <int VEC>
__device__ __forceinline__ void load_floats(const float *p, float *f) {
    if constexpr (VEC == 1) {
        f[0] = __ldg(p);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(p + i));
            f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
        }
    }
}
template <int VEC, typename T>
__device__ __forceinline__ void store_floats(T *p, const float *f) {
    if constexpr (VEC == 1) {
        qs::store1(p, f[0]);
    } else {
        qs::store_quads<VEC / 4>(p, reinterpret_cast<const float4 *>(f));
    }
}

// Sums over the threads of a row (blockDim.x of them: one warp, or whole warps with a
// named barrier of the row's own).
template <int N>
struct RowSums {
    float (*slots)[N];   // two rounds of 32
    int round = 0;
    __device__ __forceinline__ void sum(float *v) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int o = 16; o; o /= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        const int warps = blockDim.x / 32;
        if (warps == 1) return;
        // (Two sets of slots in turn: a set is written again only behind the other one's barrier.)
        float(*s)[N] = slots + round * 32;
        round ^= 1;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) s[threadIdx.x / 32][i] = v[i];
        qs::named_bar_sync(threadIdx.y + 1, blockDim.x);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += s[w][i];
    }
};

constexpr int kMostRows = 8;   // rows of a CTA

template <typename T, int VEC, int PER, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_fwd_kernel(const NormArgs a) {
    __shared__ float slots[kMostRows][64][1];
    const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= a.R) return;   // (all threads of the row)
    const T *x = static_cast<const T *>(a.x) + row * a.ld;
    Raw<T, VEC> raw[PER];
    float v[PER][VEC];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
        if (c < a.D) raw[j].load(x + c);
    }
    RowSums<1> rs{slots[threadIdx.y]};
    float m[1] = {0.f}, q[1] = {0.f};
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
        raw[j].get(v[j]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) m[0] += c < a.D ? v[j][i] : 0.f;
    }
    rs.sum(m);
    m[0] *= a.inv_d;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            v[j][i] -= m[0];
            q[0] += c < a.D ? v[j][i] * v[j][i] : 0.f;
        }
    }
    rs.sum(q);
    const float r = 1.f / sqrtf(fmaf(q[0], a.inv_d, a.eps));
    T *y = static_cast<T *>(a.y) + row * a.D;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
        if (c >= a.D) continue;
        float w[VEC], b[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[i] = 1.f, b[i] = 0.f;
        if (a.w) load_floats<VEC>(a.w + c, w);
        if (a.b) load_floats<VEC>(a.b + c, b);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = fmaf(v[j][i] * r, w[i], b[i]);
        store_floats<VEC>(y + c, v[j]);
    }
}

// A persistent CTA takes every gridDim.x-th group of rows; a thread keeps its columns, and
// with them the sums of the weights' gradients, from row to row.
template <typename T, int VEC, int PER, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_bwd_kernel(const NormArgs a) {
    __shared__ float slots[kMostRows][64][2];
    const long long stride = (long long)gridDim.x * blockDim.y;
    float w[PER][VEC], dw[PER][VEC], db[PER][VEC];
    Raw<T, VEC> rx[PER], rd[PER];
    auto fetch = [&](long long row) {
        if (row >= a.R) return;
        const T *x = static_cast<const T *>(a.x) + row * a.ld, *dy = static_cast<const T *>(a.dy) + row * a.D;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int c = (j * blockDim.x + threadIdx.x) * VEC;
            if (c < a.D) rx[j].load(x + c), rd[j].load(dy + c);
        }
    };
    long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
    fetch(row);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int c = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) w[j][i] = 1.f, dw[j][i] = db[j][i] = 0.f;
        if (a.w && c < a.D) load_floats<VEC>(a.w + c, w[j]);
    }
    RowSums<2> rs{slots[threadIdx.y]};
    for (; row < a.R; row += stride) {
        float x[PER][VEC], dy[PER][VEC], s[2] = {0.f, 0.f}, t[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int c = (j * blockDim.x + threadIdx.x) * VEC;
            rx[j].get(x[j]), rd[j].get(dy[j]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                if (c >= a.D) x[j][i] = dy[j][i] = 0.f;
                s[0] += x[j][i];
                s[1] = fmaf(dy[j][i], w[j][i], s[1]);
            }
        }
        fetch(row + stride);   // the next row's values are on their way meanwhile
        rs.sum(s);
        const float m = s[0] * a.inv_d, dn = s[1] * a.inv_d;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int c = (j * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                x[j][i] = c < a.D ? x[j][i] - m : 0.f;
                t[0] = fmaf(x[j][i], x[j][i], t[0]);
                t[1] = fmaf(dy[j][i] * w[j][i], x[j][i], t[1]);
            }
        }
        rs.sum(t);
        const float r = 1.f / sqrtf(fmaf(t[0], a.inv_d, a.eps)), dot = t[1] * r * a.inv_d;
        T *out = static_cast<T *>(a.y) + row * a.D;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int c = (j * blockDim.x + threadIdx.x) * VEC;
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float n = x[j][i] * r;
                dw[j][i] = fmaf(dy[j][i], n, dw[j][i]);
                db[j][i] += dy[j][i];
                o[i] = r * (fmaf(dy[j][i], w[j][i], -dn) - n * dot);
            }
            if (c < a.D) store_floats<VEC>(out + c, o);
        }
    }
    if (!a.part) return;
    // The CTA's rows one after the other, in place of the first one's.
    extern __shared__ float sums[];   // [2][blockDim.x * PER * VEC]
    const int n = blockDim.x * PER * VEC;
    for (int y = 0; y < (int)blockDim.y; ++y) {
        if ((int)threadIdx.y == y)
#pragma unroll
            for (int j = 0; j < PER; ++j)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const int at = (j * VEC + i) * blockDim.x + threadIdx.x;
                    sums[at] = y ? sums[at] + dw[j][i] : dw[j][i];
                    sums[n + at] = y ? sums[n + at] + db[j][i] : db[j][i];
                }
        __syncthreads();
    }
    const int threads = blockDim.x * blockDim.y, tid = threadIdx.y * blockDim.x + threadIdx.x;
    float *part = a.part + (size_t)blockIdx.x * 2 * a.D;
    for (int c = tid; c < a.D; c += threads) {
        const int v = c / VEC, at = (v / blockDim.x * VEC + c % VEC) * blockDim.x + v % blockDim.x;
        part[c] = sums[at];
        part[a.D + c] = sums[n + at];
    }
}

// dw and db: the sum of the CTAs' parts, 32 columns and 32 groups of parts per CTA.
__global__ void __launch_bounds__(1024) norm_weights_kernel(const float *part, float *dw, float *db, unsigned parts, unsigned D) {
    __shared__ float sums[32][33];
    const unsigned x = threadIdx.x % 32, y = threadIdx.x / 32, col = blockIdx.x * 32 + x;
    float s = 0.f;
    if (col < 2 * D)
        for (unsigned p = y; p < parts; p += 32) s += part[(size_t)p * 2 * D + col];
    sums[y][x] = s;
    __syncthreads();
    s = sums[x][y];   // column y of the CTA's, group x
#pragma unroll
    for (int o = 16; o; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    const unsigned c = blockIdx.x * 32 + y;
    if (x == 0 && c < 2 * D) {
        float *out = c < D ? dw : db;
        if (out) out[c < D ? c : c - D] = s;
    }
}

using Kernel = void (*)(NormArgs);

// THREADS: the most a CTA has; the register allotment goes by it (rows of more than 8192
// values, or single rows spread thin, are the ones that need 1024).
template <bool BWD, typename T, int VEC, int THREADS>
Kernel pick_per(int per) {
    if constexpr (BWD) {
        if constexpr (VEC == 8) return per <= 1 ? norm_bwd_kernel<T, VEC, 1, THREADS> : norm_bwd_kernel<T, VEC, 2, THREADS>;
        else if constexpr (VEC == 4) return per <= 2 ? norm_bwd_kernel<T, VEC, 2, THREADS> : norm_bwd_kernel<T, VEC, 4, THREADS>;
        else return per <= 4 ? norm_bwd_kernel<T, VEC, 4, THREADS> : norm_bwd_kernel<T, VEC, 16, THREADS>;
    } else {
        if constexpr (VEC == 1) return per <= 4 ? norm_fwd_kernel<T, VEC, 4, THREADS> : norm_fwd_kernel<T, VEC, 16, THREADS>;
        else return per <= 1 ? norm_fwd_kernel<T, VEC, 1, THREADS> : per <= 4 ? norm_fwd_kernel<T, VEC, 4, THREADS> : norm_fwd_kernel<T, VEC, 8, THREADS>;
    }
}
template <bool BWD>
Kernel pick(int dtype, bool wide, int per, int threads) {
    constexpr int FEW = BWD ? 512 : 256;
    if (threads <= FEW) {
        if (dtype == QS_BF16) return wide ? pick_per<BWD, __nv_bfloat16, 8, FEW>(per) : pick_per<BWD, __nv_bfloat16, 1, FEW>(per);
        return wide ? pick_per<BWD, float, 4, FEW>(per) : pick_per<BWD, float, 1, FEW>(per);
    }
    if (dtype == QS_BF16) return wide ? pick_per<BWD, __nv_bfloat16, 8, 1024>(per) : pick_per<BWD, __nv_bfloat16, 1, 1024>(per);
    return wide ? pick_per<BWD, float, 4, 1024>(per) : pick_per<BWD, float, 1, 1024>(per);
}

// Threads of a row: a power of two, 32 .. 1024, with at most `most` units of a row each.
int lanes_of(long long units, int most) {
    int n = 32;
    while ((long long)n * most < units && n < 1024) n *= 2;
    return n;
}

int check(int dtype, float eps, int64_t R, int64_t D, int64_t ld) {
    if ((dtype != QS_F32 && dtype != QS_BF16) || !(eps >= 0.f) || !(eps <= 3.4e38f)) return QS_ERR_DIMS;
    if (R < 0 || D < 0 || D > QS_NORM_MAX_D || ld < 0) return QS_ERR_DIMS;
    if (R >= int64_t(1) << 31 || ld >= int64_t(1) << 40 || (__int128)R * ld >= ((__int128)1 << 46)) return QS_ERR_DIMS;
    return R == 0 || D == 0 ? 1 : QS_OK;
}

bool skew(const void *p, int m) { return reinterpret_cast<uintptr_t>(p) % m != 0; }

int launched() { return cudaGetLastError() == cudaSuccess ? QS_OK : QS_ERR_CUDA; }

}  // namespace

extern "C" int quat_layer_norm_fwd(int dtype, float eps, const void *x, const float *w, const float *b, void *y, int64_t R,
                                   int64_t D, int64_t ld, void *stream_) {
    const int dc = check(dtype, eps, R, D, ld);
    if (dc == 1) return QS_OK;
    if (dc != QS_OK) return dc;
    if (!x || !y) return QS_ERR_NULL;
    const int es = dtype == QS_BF16 ? 2 : 4;
    if (skew(x, es) || skew(y, es) || skew(w, 4) || skew(b, 4)) return QS_ERR_MISALIGNED;
    const size_t ny = (size_t)R * D * es, nx = (size_t)((R - 1) * ld + D) * es, nw = (size_t)D * 4;
    if (qsh::overlaps(y, ny, x, nx) || qsh::overlaps(y, ny, w, nw) || qsh::overlaps(y, ny, b, nw)) return QS_ERR_ALIAS;
    int dev = 0, sms = 0;
    const int rc = qsh::device(&dev, &sms);
    if (rc != QS_OK) return rc;
    NormArgs a{};
    a.x = x, a.w = w, a.b = b, a.y = y, a.R = R, a.ld = ld, a.D = (int)D, a.eps = eps, a.inv_d = 1.f / (float)D;
    const int vec = 16 / es;
    const bool wide = D % vec == 0 && ld % vec == 0 && !qsh::misaligned(x) && !qsh::misaligned(y) && !qsh::misaligned(w) && !qsh::misaligned(b);
    const long long units = wide ? D / vec : D;
    // One warp per row of up to 8 units a lane, whose sums need no barrier; more threads where
    // rows are longer, or where there are too few rows to fill the GPU.
    int lanes = lanes_of(units, wide ? 8 : 16);
    while (lanes < 1024 && lanes < units && R * lanes < 512 * (int64_t)sms) lanes *= 2;
    const int rows = lanes >= 256 ? 1 : 256 / lanes;
    const Kernel fn = pick<false>(dtype, wide, (int)((units + lanes - 1) / lanes), lanes * rows);
    fn<<<(unsigned)((R + rows - 1) / rows), dim3(lanes, rows), 0, static_cast<cudaStream_t>(stream_)>>>(a);
    return launched();
}

extern "C" int quat_layer_norm_bwd(int dtype, float eps, const void *x, const float *w, const void *d_y, void *d_x, float *d_w,
                                   float *d_b, int64_t R, int64_t D, int64_t ld, void *stream_) {
    const int dc = check(dtype, eps, R, D, ld);
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (dc != QS_OK && dc != 1) return dc;
    if (skew(d_w, 4) || skew(d_b, 4)) return QS_ERR_MISALIGNED;
    if (dc == 1) {   // no rows: the sums over them are zero
        for (float *p : {d_w, d_b})
            if (p && D > 0 && cudaMemsetAsync(p, 0, (size_t)D * 4, stream) != cudaSuccess) {
                cudaGetLastError();
                return QS_ERR_CUDA;
            }
        return QS_OK;
    }
    if (!x || !d_y || !d_x) return QS_ERR_NULL;
    const int es = dtype == QS_BF16 ? 2 : 4;
    if (skew(x, es) || skew(d_y, es) || skew(d_x, es) || skew(w, 4)) return QS_ERR_MISALIGNED;
    const size_t n = (size_t)R * D * es, nx = (size_t)((R - 1) * ld + D) * es, nw = (size_t)D * 4;
    const struct { const void *p; size_t n; } ins[] = {{x, nx}, {w, nw}, {d_y, n}}, outs[] = {{d_x, n}, {d_w, nw}, {d_b, nw}};
    for (int i = 0; i < 3; ++i) {
        for (const auto &in : ins)
            if (qsh::overlaps(outs[i].p, outs[i].n, in.p, in.n)) return QS_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (qsh::overlaps(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return QS_ERR_ALIAS;
    }
    int dev = 0, sms = 0;
    int rc = qsh::device(&dev, &sms);
    if (rc != QS_OK) return rc;
    NormArgs a{};
    a.x = x, a.w = w, a.dy = d_y, a.y = d_x, a.R = R, a.ld = ld, a.D = (int)D, a.eps = eps, a.inv_d = 1.f / (float)D;
    const int vec = 16 / es;
    const bool wide = D % vec == 0 && ld % vec == 0 && !qsh::misaligned(x) && !qsh::misaligned(d_y) && !qsh::misaligned(d_x) && !qsh::misaligned(w);
    const long long units = wide ? D / vec : D;
    // At most 16 values a thread: with their weights, sums and the next row's they fill its registers.
    int lanes = lanes_of(units, wide ? 16 / vec : 16);
    while (lanes < 1024 && lanes < units && R * lanes < 512 * (int64_t)sms) lanes *= 2;
    const int rows = lanes >= 512 ? 1 : 512 / lanes < kMostRows ? 512 / lanes : kMostRows;
    const int per = (int)((units + lanes - 1) / lanes);
    const long long all = (R + rows - 1) / rows;
    const Kernel fn = pick<true>(dtype, wide, per, lanes * rows);
    const int slots = wide ? vec == 8 ? (per <= 1 ? 1 : 2) : (per <= 2 ? 2 : 4) : (per <= 4 ? 4 : 16);   // PER of the kernel picked
    const size_t smem = d_w || d_b ? (size_t)lanes * slots * (wide ? vec : 1) * 2 * sizeof(float) : 0;
    int fit = 1;
    if (smem > 48 * 1024 && cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return cudaGetLastError(), QS_ERR_CUDA;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, fn, lanes * rows, smem) != cudaSuccess || fit < 1) return cudaGetLastError(), QS_ERR_CUDA;
    const unsigned grid = (unsigned)(all < (long long)sms * fit ? all : (long long)sms * fit);
    qsh::Hold hold;
    if (d_w || d_b) {
        unsigned char *ws = nullptr;
        rc = qsh::workspace(dev, stream, sizeof(qs::WsHeader) + (size_t)grid * 2 * D * 4, &ws, &hold);
        if (rc != QS_OK) return rc;
        a.part = reinterpret_cast<float *>(ws + sizeof(qs::WsHeader));
    }
    fn<<<grid, dim3(lanes, rows), smem, stream>>>(a);
    rc = launched();
    if (rc != QS_OK || !a.part) return rc;
    norm_weights_kernel<<<(unsigned)(2 * D + 31) / 32, 1024, 0, stream>>>(a.part, d_w, d_b, grid, (unsigned)D);
    return launched();
}
