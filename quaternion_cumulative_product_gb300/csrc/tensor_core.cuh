// tensor_core.cuh -- fifth-generation tensor cores (tcgen05, tensor memory) for
// products of fp32 precision, as the delta rule's kernels use them.
//
// Precision.  tcgen05.mma multiplies bfloat16 values exactly and adds in fp32.
// An fp32 value x is carried as three bfloat16 terms x = x0 + x1 + x2, each the rounding
// to nearest of what the ones before it leave (|x1| <= 2^-8, |x2| <= 2^-17 of x's power of
// two, and nothing is left then), a bfloat16 input as itself.
// A product of values with terms i and j keeps the pairs i + j <= 2: what is left
// out is at most 2^-24 of the product, of either sign (rms 2^-27.4 over normal values).
// So a product costs 1 (bf16 x bf16), 3 (fp32 x bf16) or 6 (fp32 x fp32) tensor-core passes.
// Terms that are cut off instead (8 bits each) leave out eight times as much, always with
// the product's sign.  Two terms and the pairs i + j <= 1 leave out 2^-15 at most, rms 2^-17.8.
//
// Layouts.  Operands in shared memory are tiles of 64 values (128 bytes) a row
// with the 128-byte swizzle: 16-byte unit u of row r sits at unit u ^ (r % 8).
// Read along the row they are a K-major operand, read across the rows an
// MN-major one; the same bytes serve both.  Accumulators, and left operands
// that a kernel has computed, are in tensor memory, one row of the product
// (lane) per thread of a warpgroup.
#pragma once

#include "quat_common.cuh"

namespace qs {

// ---------------------------------------------------------------------------
// Tensor memory.
// ---------------------------------------------------------------------------
// All 512 columns (the CTA is alone on its SM); one whole warp calls each.
__device__ __forceinline__ void tmem_alloc_all(uint32_t *slot) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_all(uint32_t base) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define QS_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define QS_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 columns of this thread's lane (the warp's lanes are 32 * (warp % 4) ..).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : QS_R8(r, 0), QS_R8(r, 8), QS_R8(r, 16), QS_R8(r, 24)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : QS_R8(r, 0), QS_R8(r, 8)
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        QS_W8(r, 0), QS_W8(r, 8)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), QS_W8(r, 0)
                 : "memory");
}

// ---------------------------------------------------------------------------
// Descriptors and products.
// ---------------------------------------------------------------------------
// One thread of a converged warp.  Products are issued under it, with operands that
// are the same for the whole warp: their descriptors stay in uniform registers
// (under `threadIdx.x == 0` each product costs several moves to them, and 85 to 125
// clocks instead of the 64 that the tensor cores take).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ int warp_uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Shared-memory operand, 128-byte swizzle.  K-major: `sbo` = bytes between groups
// of 8 rows.  MN-major: `lbo` = bytes between blocks of 64 values along M or N,
// `sbo` = bytes between groups of 8 along K.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// Instruction descriptor: bf16 x bf16 -> fp32, M x N.
__host__ __device__ constexpr uint32_t mma_desc(int M, int N, bool a_mn = false, bool b_mn = false) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N / 8) << 17) |
           ((uint32_t)(M / 16) << 24);
}

// D[tmem] (+)= A[smem] B[smem], 16 values of K; one thread.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A's row is a lane, two values of K a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// Arrives on `bar` once the products issued so far by this thread are done.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// ---------------------------------------------------------------------------
// Splitting fp32 values into bfloat16 terms, two at a time.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Pairs of fp32 values in one instruction.
__device__ __forceinline__ float2 fma2(const float2 a, const float2 b, const float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&r))
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)), "l"(*reinterpret_cast<const unsigned long long *>(&b)),
          "l"(*reinterpret_cast<const unsigned long long *>(&c)));
    return r;
}
__device__ __forceinline__ float2 mul2(const float2 a, const float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<unsigned long long *>(&r))
        : "l"(*reinterpret_cast<const unsigned long long *>(&a)), "l"(*reinterpret_cast<const unsigned long long *>(&b)));
    return r;
}

// The terms of a pair: three hold an fp32 value as it is.  (Infinities become NaN, and so do
// values that round to one, past 2^128 - 2^119; NaNs stay.)
template <int TERMS>
__device__ __forceinline__ void split2(float2 x, uint32_t *t) {
    const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
        t[i] = pack_bf16(x.x, x.y);
        if (i < TERMS - 1) x = fma2(make_float2(__uint_as_float(t[i] << 16), __uint_as_float(t[i] & 0xffff0000u)), minus, x);
    }
}
template <int TERMS>
__device__ __forceinline__ void split2(float a, float b, uint32_t *t) {
    split2<TERMS>(make_float2(a, b), t);
}

// Byte offset of 16-byte unit u of row r in a tile of 128-byte rows.
__device__ __forceinline__ uint32_t swizzled(int r, int u) { return (uint32_t)(r * 128 + ((u ^ (r & 7)) << 4)); }

__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void *gmem, bool copy) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(copy ? 16 : 0) : "memory");
}

// ---------------------------------------------------------------------------
// Waits.  Bounded: a wait that runs out records the error and raises the CTA's
// `gone` flag, and from then on no wait of the CTA blocks.  A wait tells whether its phase
// came; a thread that issues products or copies sends no more once one of its own did
// not (a copy would arrive on a barrier that still waits for the last one).  All
// threads run on to the CTA's end, through the same barriers, on whatever they hold.  There the issuing threads wait for what is still in flight
// (drain_*, again with a limit) before the tensor memory is freed.  The outputs are then
// invalid, and quat_cumprod_status reports QS_ERR_TIMEOUT.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, volatile int *gone, const Control &ctl) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*gone) return false;
        if (global_timer_ns() - t0 > ctl.timeout_ns) {
            *gone = 1;
            record_error(ctl.hdr, (int)blockIdx.x);
            return false;
        }
    }
    return true;
}

// Waits for a phase whatever the flag says, up to the limit.
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity, const Control &ctl) {
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 <= ctl.timeout_ns) {
    }
}

// The thread that issued the products waits for them on a barrier of its own.
__device__ __forceinline__ void drain_products(uint64_t *bar, const Control &ctl) {
    mma_commit(bar);
    drain_wait(bar, 0, ctl);
}

// The same for a whole warp, converged afterwards (tensor-memory loads and stores
// want the warp's threads together).
__device__ __forceinline__ bool tc_wait_warp(uint64_t *bar, uint32_t parity, volatile int *gone, const Control &ctl) {
    const bool ok = tc_wait(bar, parity, gone, ctl);
    __syncwarp();
    tc_fence_after();
    return ok;
}

}  // namespace qs
