"""Builds libtks.so (the CUDA library) in-tree with nvcc, for sm_103a, and the C++ binding
of the cache, attention, block and page calls with the host compiler."""

from __future__ import annotations

import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libtks.so")

SOURCES = [os.path.join(CSRC, "tks_select.cu"), os.path.join(CSRC, "tks_select512.cu"),
           os.path.join(CSRC, "tks_order.cu"), os.path.join(CSRC, "tks_cache.cu"),
           os.path.join(CSRC, "tks_attn.cu"), os.path.join(CSRC, "tks_attn_rows.cu"),
           os.path.join(CSRC, "tks_attn_tiles.cu"), os.path.join(CSRC, "tks_attn_tiles_bf16.cu"),
           os.path.join(CSRC, "tks_blocks.cu"), os.path.join(CSRC, "tks_scores_tiles.cu"),
           os.path.join(CSRC, "tks_pages.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, "tks_device.cuh"), os.path.join(CSRC, "tks_kernel.cuh"),
                     os.path.join(CSRC, "tks_internal.h"), os.path.join(CSRC, "tks_attn.cuh"),
                     os.path.join(CSRC, "tks_attn_internal.h"), os.path.join(CSRC, "tks_attn_host.h"),
                     os.path.join(CSRC, "tks_tensor.cuh"), os.path.join(CSRC, "tks_scores.cuh"),
                     os.path.join(INCLUDE, "tks.h"), os.path.join(INCLUDE, "tks_attention.h"),
                     os.path.join(INCLUDE, "tks_blocks.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
]


def nvcc_path() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtks")
    return cand


def up_to_date(path: str = LIB_PATH) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(s) <= t for s in DEPENDS)


# A measurement build: the first-round histogram with warp-aggregated adds
# (match_any) instead of plain shared-memory adds, otherwise the same library.
HIST_AGGREGATE_PATH = os.path.join(BUILD_DIR, "libtks_hist_aggregate.so")


def build(force: bool = False, verbose_ptxas: bool = False, out: str = LIB_PATH,
          hist_aggregate: bool = False) -> str:
    """Compile libtks.so unless it is newer than every source; returns its path.
    hist_aggregate: the measurement build (HIST_AGGREGATE_PATH by default)."""
    if hist_aggregate and out == LIB_PATH:
        out = HIST_AGGREGATE_PATH
    if not force and up_to_date(out):
        return out
    os.makedirs(os.path.dirname(out), exist_ok=True)
    tag = f".tmp{os.getpid()}"
    nvcc = nvcc_path()
    # one process per translation unit, in parallel, then one link
    objs = [os.path.join(os.path.dirname(out), os.path.basename(src) + tag + ".o") for src in SOURCES]
    procs = []
    for src, obj in zip(SOURCES, objs):
        cmd = [nvcc, *NVCC_FLAGS, f"-I{INCLUDE}", f"-I{CSRC}", "-c", src, "-o", obj]
        if hist_aggregate:
            cmd.insert(1, "-DTKS_HIST_AGGREGATE=1")
        if verbose_ptxas:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd)))
    failed = [src for src, pr in procs if pr.wait() != 0]
    try:
        if failed:
            raise subprocess.CalledProcessError(1, f"nvcc -c {' '.join(failed)}")
        tmp = out + tag
        subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", *objs,
                        "-o", tmp], check=True)
        os.replace(tmp, out)
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
    return out


# The C++ step between Python and the cache, attention, block and page calls: an extension
# module built by the host compiler against torch's headers.
BINDING_SOURCE = os.path.join(CSRC, "tks_binding.cpp")


def binding_path() -> str:
    """Where the binding for this Python and this torch is: one built for another does not fit."""
    import sysconfig

    import torch

    tag = f"{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(BUILD_DIR, f"tks_binding.{tag}.so")


def _binding_up_to_date() -> bool:
    path = binding_path()
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(s) <= t for s in (BINDING_SOURCE, os.path.join(INCLUDE, "tks.h"),
                                                  os.path.join(INCLUDE, "tks_attention.h"),
                                                  os.path.join(INCLUDE, "tks_blocks.h")))


def start_binding(force: bool = False):
    """Starts compiling the binding unless it is up to date; finish_binding() takes what this returns."""
    if not force and _binding_up_to_date():
        return None
    import sysconfig
    import tempfile

    import torch

    os.makedirs(BUILD_DIR, exist_ok=True)
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    # (a name of its own for every build: threads and processes may come here together)
    fd, tmp = tempfile.mkstemp(prefix="tks_binding.", suffix=".tmp", dir=BUILD_DIR)
    os.close(fd)
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", BINDING_SOURCE, "-o", tmp,
           f"-I{INCLUDE}", f"-I{inc}", f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
           f"-I{os.path.join(cuda, 'include')}", f"-I{sysconfig.get_paths()['include']}",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-L{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]
    return subprocess.Popen(cmd), tmp


def finish_binding(started) -> str:
    path = binding_path()
    if started is not None:
        proc, tmp = started
        if proc.wait() != 0:
            os.remove(tmp)
            raise subprocess.CalledProcessError(proc.returncode, f"g++ {BINDING_SOURCE}")
        os.chmod(tmp, 0o755)
        os.replace(tmp, path)
    return path


def build_binding(force: bool = False) -> str:
    """Compile the binding unless it is newer than its sources; returns its path."""
    return finish_binding(start_binding(force))


if __name__ == "__main__":
    import sys
    started = start_binding("--force" in sys.argv)
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
    print(finish_binding(started))
