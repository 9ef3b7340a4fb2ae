// workspace.h -- the library's scratch memory of one (device, stream): grown to what a
// call needs.  `Gpu` makes the CUDA calls (the host tests put a fake in its place).
#pragma once

#include <cstddef>
#include <utility>
#include <vector>

#include "quat_cumprod.h"

namespace qsh {

// A capture writes the scratch's address into its graph, which may be replayed for as long
// as the program likes.  Scratch that a capture has been given is therefore kept when
// a later call outgrows it (`kept`, for the life of the process), never freed.
struct Workspace {
    unsigned char *base = nullptr;
    size_t bytes = 0;
    bool captured = false;               // a capture has been given `base`
    std::vector<unsigned char *> kept;   // outgrown, but in a graph
};

// Scratch of at least `need` bytes for a call on `stream`; new scratch starts with zeros in
// its first `head` bytes.  `Gpu`: static bool capturing(Stream, bool *), synchronize(Stream),
// allocate(size_t, unsigned char **), clear(unsigned char *, size_t, Stream), release(unsigned char *).
template <typename Gpu, typename Stream>
int ensure(Workspace &w, Stream stream, size_t need, size_t head, unsigned char **out) {
    bool capturing = false;
    if ((!w.captured || w.bytes < need) && !Gpu::capturing(stream, &capturing)) return QS_ERR_CUDA;
    if (w.bytes >= need) {
        w.captured |= capturing;
        *out = w.base;
        return QS_OK;
    }
    if (capturing) return QS_ERR_NOMEM;
    if (w.base) {
        if (!Gpu::synchronize(stream)) return QS_ERR_CUDA;
        if (w.captured) w.kept.push_back(w.base);
        else Gpu::release(w.base);
        w = {nullptr, 0, false, std::move(w.kept)};
    }
    const size_t align = size_t(1) << 20, bytes = (need + need / 4 + align - 1) / align * align;
    unsigned char *p = nullptr;
    if (!Gpu::allocate(bytes, &p)) return QS_ERR_NOMEM;
    if (!Gpu::clear(p, head, stream) || !Gpu::synchronize(stream)) {
        Gpu::release(p);
        return QS_ERR_CUDA;
    }
    w.base = p;
    w.bytes = bytes;
    *out = p;
    return QS_OK;
}

}  // namespace qsh
