"""Build the in-tree CUDA libraries for sm_103a with nvcc (no cmake): libvt_attn.so, and
libvt_attn_debug.so, the same sources with VT_DEBUG (device index checks that report
VT_ERR_DEVICE_BOUNDS).  Every translation unit of both compiles in parallel."""

from __future__ import annotations

import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libvt_attn.so")
LIB_DEBUG = os.path.join(PKG, "libvt_attn_debug.so")
SOURCES = [os.path.join(CSRC, f) for f in ("vt_attn_api.cu", "vt_qk_rope_api.cu", "vt_attn_prefix_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("vt_attn_f32_2q.cuh", "vt_attn_bf16_2q.cuh", "vt_attn_common.cuh", "vt_attn_merge.cuh",
                                                  "vt_ptx.cuh", "vt_host.h", "vt_qk_rope.cuh", "vt_attn_stream.cuh")] + [
    os.path.join(os.path.dirname(PKG), "include", "vt_attn.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-v",
]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libvt_attn.so")


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in DEPS if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libvt_attn.so and libvt_attn_debug.so next to this file; returns the release library's path."""
    jobs, links = [], []
    for lib, extra in ((LIB, []), (LIB_DEBUG, ["-DVT_DEBUG"])):
        if force or not up_to_date(lib):
            objs = [f"{lib}.{os.path.basename(src)}.o" for src in SOURCES]
            links.append((lib, objs))
            for src, obj in zip(SOURCES, objs):
                cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", "-o", obj, src]
                jobs.append((obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    results = [(obj, proc, *proc.communicate()) for obj, proc in jobs]
    for obj, proc, out, err in results:
        if proc.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(obj)} ({proc.returncode}):\n{out}\n{err}")
        if verbose:
            print(err)
    for lib, objs in links:
        tmp = lib + ".tmp"
        r = subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"linking {os.path.basename(lib)} failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
        for obj in objs:
            os.remove(obj)
    return LIB
