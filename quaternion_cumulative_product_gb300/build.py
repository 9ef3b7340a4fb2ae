"""Builds ``libquatscan.so`` (the CUDA library behind ``include/quat_cumprod.h``).

Its translation units are compiled side by side for sm_103a only and linked with
the static CUDA runtime, in place next to this file.  Used by
``__graft_entry__.build()``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", f) for f in
           ("quat_scan.cu", "norm_rotate.cu", "delta_rule.cu", "delta_step.cu", "decay.cu", "layer_norm.cu", "dropout.cu")]
HEADERS = [os.path.join(HERE, "csrc", f) for f in
           ("quat_device.cuh", "quat_common.cuh", "quat_tiles.cuh", "quat_chain.cuh", "quat_walk.cuh",
            "quat_segwalk.cuh", "quat_segwalk_ws.cuh", "quat_segwalk_bwd.cuh", "quat_segwalk_tab.cuh",
            "quat_short.cuh", "quat_host.h", "workspace.h", "mixer_device.cuh", "delta_common.cuh", "tensor_core.cuh",
            "delta_prep.cuh", "delta_fwd_tc.cuh", "delta_bwd_tc.cuh", "delta_chain_tc.cuh", "delta_host.cuh", "decay_walk.cuh", "decay_gate.cuh", "decay_states.cuh")]
DEPS = SOURCES + HEADERS + [os.path.join(ROOT, "include", f) for f in ("quat_cumprod.h", "quat_mixer.h", "quat_block.h")]
LIB = os.path.join(HERE, "libquatscan.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (CUDA toolkit required to build libquatscan.so)")


def command(source: str, out: str, extra=()) -> list:
    """Compiles one translation unit to an object file."""
    return [nvcc_path(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
            "-c", "-I", os.path.join(ROOT, "include"), *extra, source, "-o", out]


def link_command(objects, out: str) -> list:
    return [nvcc_path(), *ARCH, "-shared", "-Xcompiler", "-fPIC", *objects, "-o", out]


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in DEPS)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not is_stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    extra = ("-Xptxas", "-v") if verbose else ()

    def run(cmd):
        proc = subprocess.run(cmd, capture_output=True, text=True)
        if proc.returncode != 0:
            sys.stderr.write(proc.stdout + proc.stderr)
            raise RuntimeError("nvcc failed to build libquatscan.so")
        return proc.stderr

    with tempfile.TemporaryDirectory() as objdir, ThreadPoolExecutor(len(SOURCES)) as pool:
        objects = [os.path.join(objdir, os.path.basename(s) + ".o") for s in SOURCES]
        said = list(pool.map(lambda so: run(command(*so, extra)), zip(SOURCES, objects)))
        run(link_command(objects, tmp))
    if verbose:
        sys.stderr.write("".join(said))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
