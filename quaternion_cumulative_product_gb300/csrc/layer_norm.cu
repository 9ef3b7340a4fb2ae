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
// by 4 .. 1024 threads (a power of two), 16 bytes to an access where rows and pointers
// are aligned so, single values (neighbouring lanes neighbouring values) where not.  CTAs are
// persistent: a thread keeps its columns' weights (and, backward, the sums of their gradients)
// from row to row, because weights read from the L1 cache for every row are twice a bfloat16
// row's own bytes, and the next row's values are on their way while one is worked on.  Long
// batches of rows up to 2048 (bfloat16) or 1024 (fp32) values go forward by a warp per row, whose
// sums need no barrier.
#include <algorithm>
#include <type_traits>

#include "mixer_device.cuh"
#include "quat_common.cuh"
#include "quat_block.h"
#include "quat_host.h"
#include "tensor_core.cuh"   // fma2, mul2

namespace {

struct NormArgs {
    const void *x, *dy;
    const float *w, *b;
    void *y;       // y; backward: d_x
    float *part;   // backward: sums of each CTA [grid][2][D]
    long long R, ld;
    int D;
    float eps, inv_d;
    qs::Control ctl;
};

// VEC values as they are in memory.
template <typename T, int VEC>
struct Raw;
template <>
struct Raw<float, 4> {
    float4 r;
    __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float *p) { r = __ldg(reinterpret_cast<const float4 *>(p)); }
    __device__ __forceinline__ void shared(const float *p) { r = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void get(float *f) const { f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w; }
};
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 r;
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void shared(const __nv_bfloat16 *p) { r = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float *f) const {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(u[i] << 16), f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
};
template <typename T>
struct Raw<T, 1> {
    T r;
    __device__ __forceinline__ void zero() { r = T(0.f); }
    __device__ __forceinline__ void load(const T *p) { r = *p; }
    __device__ __forceinline__ void get(float *f) const { f[0] = qs::to_float(r); }
};


__device__ __forceinline__ float2 add2(const float2 a, const float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&r))
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)), "l"(*reinterpret_cast<const unsigned long long *>(&b)));
    return r;
}

// The arithmetic on pairs of values, and on single ones.
__device__ __forceinline__ float add2(float a, float b) { return a + b; }
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 mul2(const float2 a, const float2 b) { return qs::mul2(a, b); }
__device__ __forceinline__ float2 fma2(const float2 a, const float2 b, const float2 c) { return qs::fma2(a, b, c); }
template <typename V>
__device__ __forceinline__ V both(float v) {
    if constexpr (sizeof(V) == 8) return make_float2(v, v);
    else return v;
}
__device__ __forceinline__ float total(float v) { return v; }
__device__ __forceinline__ float total(const float2 v) { return v.x + v.y; }

// N values: pairs, or a single one.
template <int N>
struct Vals {
    using V = std::conditional_t<N == 1, float, float2>;
    static constexpr int P = (N + 1) / 2;
    V p[P];
    __device__ __forceinline__ void fill(float v) {
#pragma unroll
        for (int i = 0; i < P; ++i) p[i] = both<V>(v);
    }
    template <typename R>
    __device__ __forceinline__ void get(const R &raw) {
        raw.get(reinterpret_cast<float *>(p));
    }
    __device__ __forceinline__ float at(int i) const { return reinterpret_cast<const float *>(p)[i]; }
    __device__ __forceinline__ void load(const float *src) {
        float *f = reinterpret_cast<float *>(p);
        if constexpr (N == 1) f[0] = __ldg(src);
        else
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(src + i));
                f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
            }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *dst) const {
        if constexpr (N == 1) qs::store1(dst, p[0]);
        else qs::store_quads<N / 4>(dst, reinterpret_cast<const float4 *>(p));
    }
};

// Sums over the threads of a row: part of a warp, one warp, or whole warps (LANES > 32, by way of
// shared memory and a named barrier of the row's own).
template <int N>
struct RowSums {
    float (*slots)[N];   // two rounds of 32
    int round = 0;
    __device__ __forceinline__ void sum(float *v) {
        const int lanes = blockDim.x;
#pragma unroll
        for (int o = 16; o; o /= 2)
            if (o < lanes)
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (lanes <= 32) return;
        const int warps = lanes / 32;
        // (Two sets of slots in turn: a set is written again only behind the other one's barrier.)
        float(*s)[N] = slots + round * 32;
        round ^= 1;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) s[threadIdx.x / 32][i] = v[i];
        qs::named_bar_sync(threadIdx.y + 1, lanes);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += s[w][i];
    }
};

constexpr int kMostRows = 128, kMostWide = 8;   // rows of a CTA; with more than one warp each

// A persistent CTA takes every gridDim.x-th group of blockDim.y rows, with blockDim.x threads each.
template <typename T, int VEC, int PER, int THREADS, bool BWD>
__global__ void __launch_bounds__(THREADS, 1) norm_kernel(const NormArgs a) {
    __shared__ float slots[kMostWide][64][2];
    const long long stride = (long long)gridDim.x * blockDim.y;
    const int lanes = blockDim.x;
    if (BWD) qs::let_next_start();
    Vals<VEC> w[PER], b[PER], dw[PER];   // backward: b holds db
    Raw<T, VEC> rx[PER], rd[PER];
    bool on[PER];
    auto fetch = [&](long long row) {
        if (row >= a.R) return;
        const T *x = static_cast<const T *>(a.x) + row * a.ld, *dy = static_cast<const T *>(a.dy) + row * a.D;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (on[j]) {
                const int c = (j * lanes + threadIdx.x) * VEC;
                rx[j].load(x + c);
                if (BWD) rd[j].load(dy + c);
            }
    };
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        on[j] = (j * lanes + (int)threadIdx.x) * VEC < a.D;
        rx[j].zero();
        if (BWD) rd[j].zero();
    }
    long long first = (long long)blockIdx.x * blockDim.y;
    fetch(first + threadIdx.y);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int c = (j * lanes + threadIdx.x) * VEC;
        w[j].fill(1.f), b[j].fill(0.f);
        if (BWD) dw[j].fill(0.f);
        if (a.w && on[j]) w[j].load(a.w + c);
        if (!BWD && a.b && on[j]) b[j].load(a.b + c);
    }
    constexpr int NS = BWD ? 2 : 1;
    RowSums<NS> rs{reinterpret_cast<float(*)[NS]>(slots[lanes > 32 ? threadIdx.y : 0])};
    for (; first < a.R; first += stride) {   // (the CTA's threads stay together)
        const long long row = first + threadIdx.y;
        Vals<VEC> x[PER], dy[PER];
        using V = typename Vals<VEC>::V;
        V s = both<V>(0.f), sd = s, t = s, td = s;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            x[j].get(rx[j]);
            if (BWD) dy[j].get(rd[j]);
#pragma unroll
            for (int i = 0; i < Vals<VEC>::P; ++i) {
                s = add2(s, x[j].p[i]);
                if (BWD) sd = fma2(dy[j].p[i], w[j].p[i], sd);
            }
        }
        fetch(row + stride);   // the next row's values are on their way meanwhile
        float u[NS];
        u[0] = total(s);
        if (BWD) u[NS - 1] = total(sd);
        rs.sum(u);
        const float m = u[0] * a.inv_d, dn = BWD ? u[NS - 1] * a.inv_d : 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (on[j])
#pragma unroll
                for (int i = 0; i < Vals<VEC>::P; ++i) {
                    x[j].p[i] = add2(x[j].p[i], both<V>(-m));
                    t = fma2(x[j].p[i], x[j].p[i], t);
                    if (BWD) td = fma2(mul2(dy[j].p[i], w[j].p[i]), x[j].p[i], td);
                }
        u[0] = total(t);
        if (BWD) u[NS - 1] = total(td);
        rs.sum(u);
        const float r = 1.f / sqrtf(fmaf(u[0], a.inv_d, a.eps));
        const float dot = BWD ? u[NS - 1] * r * a.inv_d : 0.f;
        T *out = static_cast<T *>(a.y) + row * a.D;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (!on[j] || row >= a.R) continue;
            Vals<VEC> o;
#pragma unroll
            for (int i = 0; i < Vals<VEC>::P; ++i) {
                const V n = mul2(x[j].p[i], both<V>(r));
                if constexpr (BWD) {
                    dw[j].p[i] = fma2(dy[j].p[i], n, dw[j].p[i]);
                    b[j].p[i] = add2(b[j].p[i], dy[j].p[i]);
                    const V d = fma2(dy[j].p[i], w[j].p[i], both<V>(-dn));
                    o.p[i] = mul2(fma2(n, both<V>(-dot), d), both<V>(r));
                } else {
                    o.p[i] = fma2(n, w[j].p[i], b[j].p[i]);
                }
            }
            o.store(out + (j * lanes + threadIdx.x) * VEC);
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
        // The CTA's rows one after the other, in place of the first one's.
        extern __shared__ float sums[];   // [2][lanes * PER * VEC]
        const int n = lanes * PER * VEC;
        for (int y = 0; y < (int)blockDim.y; ++y) {
            if ((int)threadIdx.y == y)
#pragma unroll
                for (int j = 0; j < PER; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int at = (j * VEC + i) * lanes + threadIdx.x;
                        const float p = dw[j].at(i), q = b[j].at(i);
                        sums[at] = y ? sums[at] + p : p;
                        sums[n + at] = y ? sums[n + at] + q : q;
                    }
            __syncthreads();
        }
        const int threads = lanes * blockDim.y, tid = threadIdx.y * lanes + threadIdx.x;
        float *part = a.part + (size_t)blockIdx.x * 2 * a.D;
        for (int c = tid; c < a.D; c += threads) {
            const int v = c / VEC, at = (v / lanes * VEC + c % VEC) * lanes + v % lanes;
            part[c] = sums[at];
            part[a.D + c] = sums[n + at];
        }
    }
}

// Forward, a warp per row of 16-byte units, PER of them a lane: no barriers.  The weights lie in
// shared memory, the next row's units wait in registers.
template <typename T, int VEC, int PER>
__global__ void __launch_bounds__(256, 2) norm_warp_kernel(const NormArgs a) {
    extern __shared__ __align__(16) float wb[];   // [w, b][32 * PER * VEC], a lane's four values beside its neighbours'
    const int lane = threadIdx.x % 32, warps = 8;
    constexpr int N = 32 * PER * VEC;
    for (int i = threadIdx.x; i < 2 * a.D; i += 256) {
        const int c = i % a.D, which = i / a.D, u = c / VEC, q = c % VEC / 4;
        const float *src = which ? a.b : a.w;
        wb[which * N + ((u / 32 * (VEC / 4) + q) * 32 + u % 32) * 4 + c % 4] = src ? src[c] : which ? 0.f : 1.f;
    }
    const long long stride = (long long)gridDim.x * warps;
    long long row = (long long)blockIdx.x * warps + threadIdx.x / 32;
    Raw<T, VEC> raw[PER];
    auto fetch = [&](long long r) {
        if (r >= a.R) return;
        const T *x = static_cast<const T *>(a.x) + r * a.ld;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if ((j * 32 + lane) * VEC < a.D) raw[j].load(x + (j * 32 + lane) * VEC);
    };
#pragma unroll
    for (int j = 0; j < PER; ++j) raw[j].zero();
    fetch(row);
    __syncthreads();
    for (; row < a.R; row += stride) {
        Raw<T, VEC> cur[PER];   // (packed, and unpacked for each of the three passes: 64 floats a lane do not fit beside the next row's)
        Vals<VEC> x;
        float2 s = make_float2(0.f, 0.f), t = s;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            cur[j] = raw[j];
            x.get(cur[j]);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) s = add2(s, x.p[i]);
        }
        fetch(row + stride);
        float m = s.x + s.y;
#pragma unroll
        for (int o = 16; o; o /= 2) m += __shfl_xor_sync(0xffffffffu, m, o);
        m *= a.inv_d;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if ((j * 32 + lane) * VEC < a.D) {
                x.get(cur[j]);
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    x.p[i] = add2(x.p[i], make_float2(-m, -m));
                    t = fma2(x.p[i], x.p[i], t);
                }
            }
        float q = t.x + t.y;
#pragma unroll
        for (int o = 16; o; o /= 2) q += __shfl_xor_sync(0xffffffffu, q, o);
        const float r = 1.f / sqrtf(fmaf(q, a.inv_d, a.eps));
        T *y = static_cast<T *>(a.y) + row * a.D;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if ((j * 32 + lane) * VEC >= a.D) continue;
            x.get(cur[j]);
#pragma unroll
            for (int k = 0; k < VEC / 4; ++k) {
                const float4 w = *reinterpret_cast<const float4 *>(wb + ((j * (VEC / 4) + k) * 32 + lane) * 4);
                const float4 b = *reinterpret_cast<const float4 *>(wb + N + ((j * (VEC / 4) + k) * 32 + lane) * 4);
                const float2 lo = mul2(add2(x.p[2 * k], make_float2(-m, -m)), make_float2(r, r)), hi = mul2(add2(x.p[2 * k + 1], make_float2(-m, -m)), make_float2(r, r));
                x.p[2 * k] = fma2(lo, make_float2(w.x, w.y), make_float2(b.x, b.y));
                x.p[2 * k + 1] = fma2(hi, make_float2(w.z, w.w), make_float2(b.z, b.w));
            }
            x.store(y + (j * 32 + lane) * VEC);
        }
    }
}

// A bounded wait (quat_common.cuh): false once the limit is past, and the outputs are then invalid.
__device__ __forceinline__ bool rows_wait(uint64_t *bar, uint32_t phase, const qs::Control &ctl) {
    if (qs::mbar_try_wait(bar, phase)) return true;
    const unsigned long long t0 = qs::global_timer_ns();
    while (!qs::mbar_try_wait(bar, phase))
        if (qs::global_timer_ns() - t0 > ctl.timeout_ns) {
            qs::record_error(ctl.hdr, (int)blockIdx.x);
            return false;
        }
    return true;
}

// Copies `bytes` (a multiple of 16, both ends 16-byte aligned) to shared memory; `bar` counts them.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(qs::smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(qs::smem_addr(bar))
                 : "memory");
}

// Backward of aligned fp32 rows, 16 / WPR of them at a time: bulk copies bring the tiles into a ring of
// three; WPR warps take a row's four sums (each lane four units, as they are in memory); then
// each thread takes four columns (PB times) of all rows, and keeps their weights and sums.  A
// row's threads meet at three barriers a tile instead of two a row: 123 instead of 148 us at 32768 x 2048.
constexpr int kTileThreads = 512, kTileStages = 3, kTileUnits = 4;   // units of a lane

template <int WPR, int PB>
__global__ void __launch_bounds__(kTileThreads, 1) norm_tile_kernel(const NormArgs a) {
    using T = float;
    constexpr int RT = 16 / WPR, UNITS = kTileUnits, VEC = 4;
    __shared__ uint64_t full[kTileStages];
    __shared__ __align__(16) float stats[RT][4], slots[2][16][2];   // (read four and two at a time)
    extern __shared__ __align__(16) unsigned char dynamic[];
    const int D = a.D, tid = threadIdx.x, warp = tid / 32, lane = tid % 32, mine = warp / WPR, part = warp % WPR;
    const uint32_t rowb = (uint32_t)D * sizeof(T), stageb = 2 * RT * rowb;
    const long long tiles = (a.R + RT - 1) / RT;
    bool ok = true;
    int sent = 0, seen = 0;
    qs::let_next_start();
    auto send = [&](long long tile) {   // thread 0
        if (tile >= tiles || !ok) return;
        unsigned char *to = dynamic + (size_t)(sent % kTileStages) * stageb;
        uint64_t *bar = &full[sent % kTileStages];
        const long long row = tile * RT;
        const int rows = (int)(a.R - row < RT ? a.R - row : RT);
        qs::mbar_arrive_expect_tx(bar, 2 * rows * rowb);
        const T *x = static_cast<const T *>(a.x) + row * a.ld;
        if (a.ld == D) bulk_load(to, x, rows * rowb, bar);
        else
            for (int i = 0; i < rows; ++i) bulk_load(to + i * rowb, x + i * a.ld, rowb, bar);
        bulk_load(to + RT * rowb, static_cast<const T *>(a.dy) + row * D, rows * rowb, bar);
        ++sent;
    };
    if (tid == 0) {
        for (int i = 0; i < kTileStages; ++i) qs::mbar_init(&full[i], 1);
        qs::fence_mbar_init();
        for (int i = 0; i < kTileStages; ++i) send(blockIdx.x + (long long)i * gridDim.x);
    }
    // A lane's columns are the same for every tile, first and second time: their weights stay with it.
    Vals<VEC> wa[UNITS];
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
        const int c = ((part * UNITS + j) * 32 + lane) * VEC;
        wa[j].fill(1.f);
        if (a.w && c < D) wa[j].load(a.w + c);
    }
    float4 wb[PB], dw[PB], db[PB];
#pragma unroll
    for (int p = 0; p < PB; ++p) {
        const int c = (p * kTileThreads + tid) * 4;
        dw[p] = db[p] = qs::q_zero(), wb[p] = make_float4(1.f, 1.f, 1.f, 1.f);
        if (a.w && c < D) wb[p] = __ldg(reinterpret_cast<const float4 *>(a.w + c));
    }
    __syncthreads();
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int st = seen % kTileStages;
        if (ok) ok = rows_wait(&full[st], (seen / kTileStages) & 1, a.ctl);
        ++seen;
        __syncwarp();
        const T *xs = reinterpret_cast<const T *>(dynamic + (size_t)st * stageb), *ds = xs + RT * D;
        const int rows = (int)(a.R - tile * RT < RT ? a.R - tile * RT : RT);
        {   // sums of this warp's share of its row
            Raw<T, VEC> rx[UNITS], rd[UNITS];
            float2 s = make_float2(0.f, 0.f), sd = s, t = s, td = s;
            const bool live = mine < rows;
#pragma unroll
            for (int j = 0; j < UNITS; ++j) {
                const int c = ((part * UNITS + j) * 32 + lane) * VEC;
                rx[j].zero(), rd[j].zero();
                if (live && c < D) {
                    rx[j].shared(xs + mine * D + c), rd[j].shared(ds + mine * D + c);
                    Vals<VEC> x, d;
                    x.get(rx[j]), d.get(rd[j]);
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        s = add2(s, x.p[i]);
                        sd = fma2(d.p[i], wa[j].p[i], sd);
                    }
                }
            }
            auto row_sum = [&](float2 &u, int round) {   // of a pair of sums
#pragma unroll
                for (int o = 16; o; o /= 2) u.x += __shfl_xor_sync(0xffffffffu, u.x, o), u.y += __shfl_xor_sync(0xffffffffu, u.y, o);
                if constexpr (WPR > 1) {
                    if (lane == 0) slots[round][warp][0] = u.x, slots[round][warp][1] = u.y;
                    qs::named_bar_sync(1 + mine, WPR * 32);
                    u = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < WPR; ++i) u = add2(u, *reinterpret_cast<const float2 *>(slots[round][mine * WPR + i]));
                }
            };
            float2 u = make_float2(total(s), total(sd));
            row_sum(u, 0);
            const float m = u.x * a.inv_d, dn = u.y * a.inv_d;
#pragma unroll
            for (int j = 0; j < UNITS; ++j) {
                const int c = ((part * UNITS + j) * 32 + lane) * VEC;
                if (live && c < D) {
                    Vals<VEC> x, d;
                    x.get(rx[j]), d.get(rd[j]);
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        const float2 y = add2(x.p[i], make_float2(-m, -m));
                        t = fma2(y, y, t);
                        td = fma2(mul2(d.p[i], wa[j].p[i]), y, td);
                    }
                }
            }
            u = make_float2(total(t), total(td));
            row_sum(u, 1);
            const float r = 1.f / sqrtf(fmaf(u.x, a.inv_d, a.eps));
            if (part == 0 && lane == 0) stats[mine][0] = m, stats[mine][1] = r, stats[mine][2] = dn, stats[mine][3] = u.y * r * a.inv_d;
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < PB; ++p) {
            const int c = (p * kTileThreads + tid) * 4;
            if (c >= D) continue;
            const float2 wl = make_float2(wb[p].x, wb[p].y), wh = make_float2(wb[p].z, wb[p].w);
            float2 wx = make_float2(dw[p].x, dw[p].y), wz = make_float2(dw[p].z, dw[p].w), bx = make_float2(db[p].x, db[p].y), bz = make_float2(db[p].z, db[p].w);
            T *out = static_cast<T *>(a.y) + tile * RT * D + c;
#pragma unroll 4
            for (int i = 0; i < rows; ++i) {
                const float4 st4 = *reinterpret_cast<const float4 *>(stats[i]);
                const float4 xv = *reinterpret_cast<const float4 *>(xs + i * D + c), dv = *reinterpret_cast<const float4 *>(ds + i * D + c);
                const float2 m2 = make_float2(-st4.x, -st4.x), r2 = make_float2(st4.y, st4.y), dn2 = make_float2(-st4.z, -st4.z), dot2 = make_float2(-st4.w, -st4.w);
                const float2 nl = mul2(add2(make_float2(xv.x, xv.y), m2), r2), nh = mul2(add2(make_float2(xv.z, xv.w), m2), r2);
                const float2 dl = make_float2(dv.x, dv.y), dh = make_float2(dv.z, dv.w);
                wx = fma2(dl, nl, wx), wz = fma2(dh, nh, wz), bx = add2(bx, dl), bz = add2(bz, dh);
                const float2 ol = mul2(fma2(nl, dot2, fma2(dl, wl, dn2)), r2), oh = mul2(fma2(nh, dot2, fma2(dh, wh, dn2)), r2);
                qs::store4(out + (size_t)i * D, make_float4(ol.x, ol.y, oh.x, oh.y));
            }
            dw[p] = make_float4(wx.x, wx.y, wz.x, wz.y), db[p] = make_float4(bx.x, bx.y, bz.x, bz.y);
        }
        __syncthreads();   // the tile and its sums are done with
        if (tid == 0) send(tile + (long long)kTileStages * gridDim.x);
    }
    if (tid == 0 && !ok)   // a wait ran out: copies may still be in flight
        for (int i = sent > kTileStages ? sent - kTileStages : 0; i < sent; ++i) rows_wait(&full[i % kTileStages], (i / kTileStages) & 1, a.ctl);
    if (!a.part) return;
    float *part_out = a.part + (size_t)blockIdx.x * 2 * D;
#pragma unroll
    for (int p = 0; p < PB; ++p) {
        const int c = (p * kTileThreads + tid) * 4;
        if (c < D) qs::store4(part_out + c, dw[p]), qs::store4(part_out + D + c, db[p]);
    }
}

// The same for bfloat16, whose conversions cost most there: WPR warps keep a row in fp32 registers from its
// first sum to its gradient, and their columns' weights and sums from row to row.  256 threads, for the
// registers; the rows come from the same kind of ring, 8 / WPR to a tile.  32768 x 2048: 79.5 us, 0.75 of a
// copy's rate (as fp32 rows, every value converted twice and read twice: 84.6; 8192 x 8192: 88 and 104; 65536 x
// 768: 76.5 and 74.4).
constexpr int kRowThreads = 256, kRowStages = 4;

template <int WPR>
__global__ void __launch_bounds__(kRowThreads, 1) norm_row_kernel(const NormArgs a) {
    using T = __nv_bfloat16;
    constexpr int RT = 8 / WPR, UNITS = kTileUnits, VEC = 8, P = UNITS * VEC / 2;   // pairs of values of a lane
    __shared__ uint64_t full[kRowStages];
    __shared__ __align__(16) float slots[2][8][2];
    extern __shared__ __align__(16) unsigned char dynamic[];
    const int D = a.D, tid = threadIdx.x, warp = tid / 32, lane = tid % 32, mine = warp / WPR, part = warp % WPR;
    const uint32_t rowb = (uint32_t)D * sizeof(T), stageb = 2 * RT * rowb;
    const long long tiles = (a.R + RT - 1) / RT;
    bool ok = true;
    int sent = 0, seen = 0;
    qs::let_next_start();
    auto send = [&](long long tile) {   // thread 0
        if (tile >= tiles || !ok) return;
        unsigned char *to = dynamic + (size_t)(sent % kRowStages) * stageb;
        uint64_t *bar = &full[sent % kRowStages];
        const long long row = tile * RT;
        const int rows = (int)(a.R - row < RT ? a.R - row : RT);
        qs::mbar_arrive_expect_tx(bar, 2 * rows * rowb);
        const T *x = static_cast<const T *>(a.x) + row * a.ld;
        if (a.ld == D) bulk_load(to, x, rows * rowb, bar);
        else
            for (int i = 0; i < rows; ++i) bulk_load(to + i * rowb, x + i * a.ld, rowb, bar);
        bulk_load(to + RT * rowb, static_cast<const T *>(a.dy) + row * D, rows * rowb, bar);
        ++sent;
    };
    if (tid == 0) {
        for (int i = 0; i < kRowStages; ++i) qs::mbar_init(&full[i], 1);
        qs::fence_mbar_init();
        for (int i = 0; i < kRowStages; ++i) send(blockIdx.x + (long long)i * gridDim.x);
    }
    const int c0 = part * UNITS * 32 * VEC + lane * VEC;   // this lane's columns: c0 + 256 j ..
    float2 w[P], dw[P], db[P];
#pragma unroll
    for (int j = 0; j < UNITS; ++j) {
        Vals<VEC> v;
        v.fill(1.f);
        if (a.w && c0 + 256 * j < D) v.load(a.w + c0 + 256 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[j * 4 + i] = v.p[i], dw[j * 4 + i] = db[j * 4 + i] = make_float2(0.f, 0.f);
    }
    __syncthreads();
    for (long long tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int st = seen % kRowStages;
        if (ok) ok = rows_wait(&full[st], (seen / kRowStages) & 1, a.ctl);
        ++seen;
        __syncwarp();
        const T *xs = reinterpret_cast<const T *>(dynamic + (size_t)st * stageb) + mine * D, *ds = xs + RT * D;
        const long long row = tile * RT + mine;
        const bool live = row < a.R;
        float2 x[P], d[P], s = make_float2(0.f, 0.f), sd = s, t = s, td = s;
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            Raw<T, VEC> rx, rd;
            rx.zero(), rd.zero();
            if (live && c0 + 256 * j < D) rx.shared(xs + c0 + 256 * j), rd.shared(ds + c0 + 256 * j);
            rx.get(reinterpret_cast<float *>(x + j * 4)), rd.get(reinterpret_cast<float *>(d + j * 4));
#pragma unroll
            for (int i = j * 4; i < j * 4 + 4; ++i) s = add2(s, x[i]), sd = fma2(d[i], w[i], sd);
        }
        __syncthreads();   // the tile has been read
        if (tid == 0) send(tile + (long long)kRowStages * gridDim.x);
        auto row_sum = [&](float &u, float &v, int round) {
#pragma unroll
            for (int o = 16; o; o /= 2) u += __shfl_xor_sync(0xffffffffu, u, o), v += __shfl_xor_sync(0xffffffffu, v, o);
            if constexpr (WPR > 1) {
                if (lane == 0) slots[round][warp][0] = u, slots[round][warp][1] = v;
                qs::named_bar_sync(1 + mine, WPR * 32);
                u = v = 0.f;
#pragma unroll
                for (int i = 0; i < WPR; ++i) u += slots[round][mine * WPR + i][0], v += slots[round][mine * WPR + i][1];
            }
        };
        float u = total(s), v = total(sd);
        row_sum(u, v, 0);
        const float m = u * a.inv_d, dn = v * a.inv_d;
#pragma unroll
        for (int j = 0; j < UNITS; ++j)
            if (c0 + 256 * j < D)
#pragma unroll
                for (int i = j * 4; i < j * 4 + 4; ++i) {
                    x[i] = add2(x[i], make_float2(-m, -m));
                    t = fma2(x[i], x[i], t);
                    td = fma2(mul2(d[i], w[i]), x[i], td);
                }
        u = total(t), v = total(td);
        row_sum(u, v, 1);
        const float r = 1.f / sqrtf(fmaf(u, a.inv_d, a.eps)), dot = v * r * a.inv_d;
        if (live) {
            T *out = static_cast<T *>(a.y) + row * D;
#pragma unroll
            for (int j = 0; j < UNITS; ++j)
                if (c0 + 256 * j < D) {
                    Vals<VEC> o;
#pragma unroll
                    for (int i = j * 4; i < j * 4 + 4; ++i) {
                        const float2 n = mul2(x[i], make_float2(r, r));
                        dw[i] = fma2(d[i], n, dw[i]), db[i] = add2(db[i], d[i]);
                        o.p[i - j * 4] = mul2(fma2(n, make_float2(-dot, -dot), fma2(d[i], w[i], make_float2(-dn, -dn))), make_float2(r, r));
                    }
                    o.store(out + c0 + 256 * j);
                }
        }
    }
    if (tid == 0 && !ok)   // a wait ran out: copies may still be in flight
        for (int i = sent > kRowStages ? sent - kRowStages : 0; i < sent; ++i) rows_wait(&full[i % kRowStages], (i / kRowStages) & 1, a.ctl);
    if (!a.part) return;
    // The rows' groups one after the other, in the ring's place.
    float *sums = reinterpret_cast<float *>(dynamic), *out = a.part + (size_t)blockIdx.x * 2 * D;
    for (int y = 0; y < RT; ++y) {
        __syncthreads();
        if (mine == y)
#pragma unroll
            for (int j = 0; j < UNITS; ++j)
                if (c0 + 256 * j < D)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int c = c0 + 256 * j + i;
                        const float p = reinterpret_cast<const float *>(dw)[j * VEC + i], q = reinterpret_cast<const float *>(db)[j * VEC + i];
                        sums[c] = y ? sums[c] + p : p, sums[D + c] = y ? sums[D + c] + q : q;
                    }
    }
    __syncthreads();
    for (int c = tid; c < 2 * D; c += kRowThreads) out[c] = sums[c];
}

// dw and db: the sum of the CTAs' parts, 32 columns and 32 groups of parts per CTA.
__global__ void __launch_bounds__(1024) norm_weights_kernel(const float *part, float *dw, float *db, unsigned parts, unsigned D) {
    __shared__ float sums[32][33];
    qs::wait_for_last();
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

// Dynamic shared memory of norm_kernel, at most: one limit for all sizes, which calls at once on several threads do not take from each other.
constexpr int kMostSums = QS_NORM_MAX_D * 2 * (int)sizeof(float);

// Values per thread, 16 forward and 8 backward (16 of bfloat16, whose next row waits packed):
// what the registers of 512 threads hold.  THREADS: rows of more than that many threads have 1024.
template <typename T, int VEC, bool BWD>
constexpr int kPer = VEC == 8 ? 2 : VEC == 4 ? (BWD ? 2 : 4) : (BWD ? 8 : 16);

template <typename T, int VEC, bool BWD>
Kernel pick_per(int per, int threads) {
    constexpr int MOST = kPer<T, VEC, BWD>, FEW = VEC == 1 ? MOST / 4 : 1;
    if (threads <= 512) return per <= FEW ? norm_kernel<T, VEC, FEW, 512, BWD> : norm_kernel<T, VEC, MOST, 512, BWD>;
    if constexpr (1024 * VEC * MOST < QS_NORM_MAX_D)   // (else 1024 threads hold the longest row)
        if (per > MOST) return norm_kernel<T, VEC, 2 * MOST, 1024, BWD>;
    return norm_kernel<T, VEC, MOST, 1024, BWD>;
}
template <bool BWD>
Kernel pick(int dtype, bool wide, int per, int threads, int *slots) {
    const int vec = wide ? dtype == QS_BF16 ? 8 : 4 : 1;
    const int most = vec == 8 ? 2 : vec == 4 ? (BWD ? 2 : 4) : (BWD ? 8 : 16), few = vec == 1 ? most / 4 : 1;
    *slots = threads <= 512 ? per <= few ? few : most : per <= most ? most : 2 * most;   // PER of the kernel
    if (dtype == QS_BF16) return wide ? pick_per<__nv_bfloat16, 8, BWD>(per, threads) : pick_per<__nv_bfloat16, 1, BWD>(per, threads);
    return wide ? pick_per<float, 4, BWD>(per, threads) : pick_per<float, 1, BWD>(per, threads);
}

// Threads of a row: a power of two, 4 .. 1024, with at most `most` units of a row each.
int lanes_of(long long units, int most) {
    int n = 4;
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

int weights(const NormArgs &a, float *d_w, float *d_b, unsigned parts, cudaStream_t stream) {
    const float *part = a.part;
    if (qsh::launch_next(norm_weights_kernel, (unsigned)(2 * a.D + 31) / 32, 1024, 0, stream, part, d_w, d_b, parts, (unsigned)a.D) == cudaSuccess) return QS_OK;
    cudaGetLastError();
    return QS_ERR_CUDA;
}

template <bool BWD>
int launch(NormArgs &a, int dtype, bool wide, long long units, int sms, float *d_w, float *d_b, int dev, cudaStream_t stream) {
    const int vec = wide ? dtype == QS_BF16 ? 8 : 4 : 1, most = vec == 8 ? 2 : vec == 4 ? (BWD ? 2 : 4) : (BWD ? 8 : 16);
    int lanes = lanes_of(units, most);
    while (lanes < 1024 && lanes < units && a.R * lanes < 512 * (long long)sms) lanes *= 2;   // too few rows to fill the GPU: spread thinner
    const int rows = lanes >= 512 ? 1 : lanes > 32 ? 512 / lanes : 256 / lanes < kMostRows ? 256 / lanes : kMostRows;
    const long long all = (a.R + rows - 1) / rows;
    int slots = 0, fit = 1;
    const Kernel fn = pick<BWD>(dtype, wide, (int)((units + lanes - 1) / lanes), lanes * rows, &slots);
    const size_t smem = d_w || d_b ? (size_t)lanes * slots * vec * 2 * sizeof(float) : 0;
    if (smem && cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSums) != cudaSuccess) return cudaGetLastError(), QS_ERR_CUDA;
    unsigned grid = (unsigned)all;
    if (all > sms) {   // as many CTAs as run at once
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, fn, lanes * rows, smem) != cudaSuccess || fit < 1) return cudaGetLastError(), QS_ERR_CUDA;
        if (all > (long long)sms * fit) grid = (unsigned)(sms * fit);
    }
    qsh::Hold hold;
    if (d_w || d_b) {
        unsigned char *ws = nullptr;
        const int rc = qsh::workspace(dev, stream, sizeof(qs::WsHeader) + (size_t)grid * 2 * a.D * 4, &ws, &hold);
        if (rc != QS_OK) return rc;
        a.part = reinterpret_cast<float *>(ws + sizeof(qs::WsHeader));
    }
    fn<<<grid, dim3(lanes, rows), smem, stream>>>(a);
    const int rc = launched();
    if (rc != QS_OK || !a.part) return rc;
    return weights(a, d_w, d_b, grid, stream);
}

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
    cudaStream_t stream = static_cast<cudaStream_t>(stream_);
    if (wide && units > 32 && units <= 256 && R >= 16 * (int64_t)sms) {   // a warp for each row
        auto go = [&](auto kernel, int per) {
            const size_t smem = (size_t)2 * 32 * per * vec * 4;
            kernel<<<(unsigned)std::min<int64_t>((R + 7) / 8, 2 * sms), 256, smem, stream>>>(a);
            return launched();
        };
        if (dtype == QS_BF16) return units <= 128 ? go(norm_warp_kernel<__nv_bfloat16, 8, 4>, 4) : go(norm_warp_kernel<__nv_bfloat16, 8, 8>, 8);
        return units <= 128 ? go(norm_warp_kernel<float, 4, 4>, 4) : go(norm_warp_kernel<float, 4, 8>, 8);
    }
    return launch<false>(a, dtype, wide, units, sms, nullptr, nullptr, dev, stream);
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
    // Rings of tiles where there are enough of them, and rows fit (8192 values of bfloat16, 4096 of fp32).
    const int cols = 32 * kTileUnits * vec, wpr = D <= cols ? 1 : D <= 2 * cols ? 2 : D <= 4 * cols ? 4 : 8;
    if (wide && D >= 256 && D <= 8 * cols && R >= 32 * (int64_t)sms / wpr) {
        auto go = [&](auto kernel, int threads, int stages, int rows, int most) {
            const size_t smem = (size_t)stages * 2 * rows * D * es;
            if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) return cudaGetLastError(), (int)QS_ERR_CUDA;
            unsigned char *ws = nullptr;
            qsh::Hold hold;
            int rc = qsh::workspace(dev, stream, sizeof(qs::WsHeader) + (size_t)sms * 2 * D * 4, &ws, &hold);
            if (rc != QS_OK) return rc;
            a.ctl = {reinterpret_cast<qs::WsHeader *>(ws), -1, qsh::timeout_ns()};
            if (d_w || d_b) a.part = reinterpret_cast<float *>(ws + sizeof(qs::WsHeader));
            kernel<<<(unsigned)sms, threads, smem, stream>>>(a);
            rc = launched();
            if (rc != QS_OK || !a.part) return rc;
            return weights(a, d_w, d_b, (unsigned)sms, stream);
        };
        auto tile = [&](auto kernel) { return go(kernel, kTileThreads, kTileStages, 16 / wpr, kTileStages * 2 * 16 * 32 * kTileUnits * 16); };
        auto row = [&](auto kernel) { return go(kernel, kRowThreads, kRowStages, 8 / wpr, kRowStages * 2 * 8 * 32 * kTileUnits * 16); };
        if (dtype == QS_BF16) return wpr == 1 ? row(norm_row_kernel<1>) : wpr == 2 ? row(norm_row_kernel<2>) : wpr == 4 ? row(norm_row_kernel<4>) : row(norm_row_kernel<8>);
        return wpr == 1 ? tile(norm_tile_kernel<1, 1>) : wpr == 2 ? tile(norm_tile_kernel<2, 1>) : wpr == 4 ? tile(norm_tile_kernel<4, 1>) : tile(norm_tile_kernel<8, 2>);
    }
    return launch<true>(a, dtype, wide, units, sms, d_w, d_b, dev, stream);
}
