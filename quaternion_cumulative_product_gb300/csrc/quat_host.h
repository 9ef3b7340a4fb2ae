// quat_host.h -- host-side services of the library shared by its translation
// units (defined in quat_scan.cu): device check, workspace, argument checks.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "quat_cumprod.h"
#include "workspace.h"

#define QS_HIDDEN __attribute__((visibility("hidden")))

namespace qsh {

// The current device's index and SM count; QS_ERR_DEVICE unless it is an sm_103.
QS_HIDDEN int device(int *dev, int *sms);

// The workspace of (device, stream) with at least `need` bytes; it starts with a
// qs::WsHeader, which the caller must leave in place.  It is the caller's while `hold` is: until
// the last launch that uses it is enqueued.
QS_HIDDEN int workspace(int dev, cudaStream_t stream, size_t need, unsigned char **base, Hold *hold);

// Limit of every device-side wait, in nanoseconds; the CTA that the test hook stalls (-1: none).
QS_HIDDEN unsigned long long timeout_ns();
QS_HIDDEN int stall_tile();

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

inline bool misaligned(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// A tensor [B, S, H, D] in memory: element distances between batch entries,
// steps and heads.
struct Strides {
    long long b, s, h;
};

// Strides of tensor `i` of a `strides` argument (contiguous when it is NULL).
inline Strides strides_of(const int64_t *strides, int i, int64_t S, int64_t H, int64_t D) {
    if (!strides) return {(long long)(S * H * D), (long long)(H * D), (long long)D};
    return {(long long)strides[3 * i], (long long)strides[3 * i + 1], (long long)strides[3 * i + 2]};
}

// Whether the strides are usable: no negative ones, multiples of 16 bytes.
inline bool bad_strides(const Strides &t, int elem) {
    const long long m = 16 / elem;
    return t.b < 0 || t.s < 0 || t.h < 0 || t.b % m || t.s % m || t.h % m;
}

// Whether a dimension of more than one entry has no extent in memory (an expanded
// view): tensor maps cannot hold it.
inline bool has_flat_dim(const Strides &t, int64_t B, int64_t S, int64_t H) {
    return (t.b == 0 && B > 1) || (t.s == 0 && S > 1) || (t.h == 0 && H > 1);
}

// Bytes from the first to past the last element.
inline size_t span_bytes(const Strides &t, int64_t B, int64_t S, int64_t H, int64_t D, int elem) {
    if (B <= 0 || S <= 0 || H <= 0) return 0;
    return (size_t)((B - 1) * t.b + (S - 1) * t.s + (H - 1) * t.h + D) * elem;
}

// Tensor map of a bfloat16 tensor [B, S, H, D] for boxes of 64 steps x 64 values of
// one head, 128-byte swizzle; what lies outside reads as zeros.
QS_HIDDEN int head_map(CUtensorMap *map, const void *p, const Strides &t, int64_t B, int64_t S, int64_t H, int64_t D);

}  // namespace qsh
