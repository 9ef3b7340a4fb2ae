"""The library's scratch bookkeeping (``csrc/workspace.h``) against a fake of the CUDA calls, on the CPU."""
from __future__ import annotations

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <set>
#include <thread>
#include "workspace.h"
#define CHECK(x) do { if (!(x)) { printf("%d: %s\n", __LINE__, #x); return 1; } } while (0)
struct Gpu {
    static inline bool busy = false, full = false;
    static inline std::set<void *> live, freed;
    static bool capturing(int, bool *c) { *c = busy; return true; }
    static bool synchronize(int) { return true; }
    static bool allocate(size_t n, unsigned char **p) {
        if (full) return false;
        *p = static_cast<unsigned char *>(malloc(n));
        live.insert(*p);
        return true;
    }
    static bool clear(unsigned char *p, size_t n, int) { memset(p, 0, n); return true; }
    static void release(unsigned char *p) { if (live.erase(p) != 1) abort(); freed.insert(p); }   // (not given back: addresses stay distinct)
};
using namespace qsh;
int main() {
    const size_t MB = 1 << 20;
    Workspace w;
    unsigned char *a = nullptr, *b = nullptr, *c = nullptr, *d = nullptr;
    BODY
    puts("ok");
}
"""

CASES = {
    # Scratch that only eager calls have had is freed when it is outgrown.
    "eager": """
        CHECK(ensure<Gpu>(w, 0, MB, 64, &a) == QS_OK && a && w.bytes >= MB);
        CHECK(ensure<Gpu>(w, 0, 10, 64, &b) == QS_OK && b == a);
        CHECK(ensure<Gpu>(w, 0, 9 * MB, 64, &c) == QS_OK && c != a && w.bytes >= 9 * MB);
        CHECK(Gpu::freed.count(a) && Gpu::live.count(c) && w.kept.empty());""",
    # A capture's scratch outlives growth, more than once; what only eager calls had in between does not.
    "captured": """
        CHECK(ensure<Gpu>(w, 0, MB, 64, &a) == QS_OK);
        Gpu::busy = true;
        CHECK(ensure<Gpu>(w, 0, MB, 64, &b) == QS_OK && b == a);
        Gpu::busy = false;
        CHECK(ensure<Gpu>(w, 0, 4 * MB, 64, &b) == QS_OK && b != a);
        CHECK(Gpu::live.count(a));
        CHECK(ensure<Gpu>(w, 0, 20 * MB, 64, &c) == QS_OK && Gpu::freed.count(b));
        Gpu::busy = true;
        CHECK(ensure<Gpu>(w, 0, 7, 64, &d) == QS_OK && d == c);
        Gpu::busy = false;
        CHECK(ensure<Gpu>(w, 0, 90 * MB, 64, &d) == QS_OK && Gpu::live.count(c) && Gpu::live.count(a));
        CHECK(w.kept.size() == 2 && w.kept[0] == a && w.kept[1] == c);""",
    # A capture cannot grow it, and is told so; the scratch stays as it was.
    "growth in a capture": """
        CHECK(ensure<Gpu>(w, 0, MB, 64, &a) == QS_OK);
        Gpu::busy = true;
        CHECK(ensure<Gpu>(w, 0, 9 * MB, 64, &b) == QS_ERR_NOMEM && !b);
        Gpu::busy = false;
        CHECK(ensure<Gpu>(w, 0, MB, 64, &c) == QS_OK && c == a && Gpu::freed.empty());""",
    # An allocation that fails leaves no stale address behind, and what a graph holds stays.
    "no memory": """
        CHECK(ensure<Gpu>(w, 0, MB, 64, &a) == QS_OK);
        Gpu::busy = true;
        CHECK(ensure<Gpu>(w, 0, MB, 64, &a) == QS_OK);
        Gpu::busy = false;
        Gpu::full = true;
        CHECK(ensure<Gpu>(w, 0, 9 * MB, 64, &b) == QS_ERR_NOMEM && !b && !w.base && w.bytes == 0);
        Gpu::full = false;
        CHECK(ensure<Gpu>(w, 0, 1, 64, &b) == QS_OK && b != a && Gpu::live.count(a) && !w.captured);""",
    # A second thread's call on the stream waits until the first one's launches are enqueued: it
    # neither comes between them nor frees their scratch.  A call on another stream does not wait.
    "two threads": """
        Workspaces<Gpu, int> all;
        std::atomic<bool> in{false};
        std::thread second;
        {
            Hold hold;
            CHECK(all.take(0, 1, MB, 64, &a, &hold) == QS_OK && hold.owns_lock());
            second = std::thread([&] {
                Hold mine;
                all.take(0, 1, 50 * MB, 64, &b, &mine);
                in = true;
            });
            Hold other;
            CHECK(all.take(0, 2, MB, 64, &c, &other) == QS_OK && c != a);
            std::this_thread::sleep_for(std::chrono::milliseconds(100));
            CHECK(!in && Gpu::live.count(a));
        }
        second.join();
        Hold last, none;
        CHECK(in && Gpu::freed.count(a) && all.bases(0, 1, &last)[0] == b && last.owns_lock());
        CHECK(all.bases(0, 3, &none).empty() && !none.owns_lock());""",
}


@pytest.mark.parametrize("case", CASES)
def test_workspace(tmp_path, case):
    (tmp_path / "t.cpp").write_text(FAKE.replace("BODY", CASES[case]))
    exe = tmp_path / "t"
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "quaternion_cumulative_product_gb300", "csrc"), str(tmp_path / "t.cpp"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout + out.stderr
