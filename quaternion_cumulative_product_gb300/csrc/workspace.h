// workspace.h -- the library's scratch memory, one piece per (device, stream): grown to what a
// call needs, and held by a call until its last launch is enqueued.  `Gpu` makes the CUDA
// calls (the host tests put a fake in its place).
#pragma once

#include <cstddef>
#include <map>
#include <mutex>
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
    std::mutex order;                    // held by the call that enqueues on it (Hold)
};

// A call's hold on its stream's scratch, from asking for it to enqueueing its last launch.
// Kernels of one call hand values to one another there: another host thread's call on the same
// stream must neither get between two of them nor outgrow the scratch before they are launched.
using Hold = std::unique_lock<std::mutex>;

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
        w.base = nullptr, w.bytes = 0, w.captured = false;
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

template <typename Gpu, typename Stream>
class Workspaces {
public:
    // Scratch of at least `need` bytes, held by `hold` until that goes.
    int take(int dev, Stream stream, size_t need, size_t head, unsigned char **out, Hold *hold) {
        Workspace *w;
        {
            std::lock_guard<std::mutex> lk(mu_);
            w = &all_[{dev, stream}];   // (a map's entries stay where they are)
        }
        *hold = Hold(w->order);
        return ensure<Gpu>(*w, stream, need, head, out);
    }

    // The stream's scratch and what it has outgrown but graphs still use, there while `hold` is.
    std::vector<unsigned char *> bases(int dev, Stream stream, Hold *hold) {
        Workspace *w;
        {
            std::lock_guard<std::mutex> lk(mu_);
            const auto it = all_.find({dev, stream});
            if (it == all_.end()) return {};
            w = &it->second;
        }
        *hold = Hold(w->order);
        std::vector<unsigned char *> v = w->kept;
        if (w->base) v.push_back(w->base);
        return v;
    }

private:
    std::mutex mu_;   // of the map; a workspace's own fields belong to the holder of its `order`
    std::map<std::pair<int, Stream>, Workspace> all_;
};

}  // namespace qsh
