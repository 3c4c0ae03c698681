"""Builds libkvattn.so in-tree for sm_103a with nvcc (one process per source)."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkvattn.so")
# Python extension module, linked against LIB beside it; the name says which Python it was built for
MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["api.cu", "rope_append.cu", "rotary.cu", "rotary_axes.cu", "decode.cu", "decode_window.cu", "decode_shared.cu", "decode_direct.cu", "decode_static.cu", "prefill.cu", "prefill_window.cu", "prefill_fp8.cu", "blocks.cu", "compact.cu", "allocator.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the kvattn CUDA library cannot be built")
    return cand


def _flags(extra=()):
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC, *extra]


def _stale(obj: str, deps: list[str]) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _build_marshal(force: bool, headers: list[str]) -> None:
    """The extension module that shortens some calls' marshalling.  The package does without it, so a Python without its
    headers is no error."""
    src, include = os.path.join(CSRC, "marshal.cpp"), sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")) or not (force or _stale(MARSHAL, [src, *headers, __file__])):
        return
    tmp = MARSHAL + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-I", include,
                        "-I", os.path.join(ROOT, "include"), src, "-o", tmp, "-L", PKG, "-l:libkvattn.so",
                        "-Wl,-rpath,$ORIGIN"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on marshal.cpp:\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    untagged = os.path.join(PKG, "_marshal.so")  # an earlier build's, of whatever Python
    if os.path.exists(untagged):
        os.remove(untagged)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    import platform

    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, "host_arch")
    arch = platform.machine()
    if not os.path.exists(stamp) or open(stamp).read() != arch or not os.path.exists(LIB):
        force = True      # objects from another host architecture or a missing library
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "kvattn.h"))
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        if force or _stale(o, [s, *headers, __file__]):
            cmd = [nvcc(), *_flags(extra_flags), "-c", s, "-o", o]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append((src, cmd))

    def run(job):
        src, cmd = job
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return src, r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, len(jobs))) as ex:
        for src, err in ex.map(run, jobs):
            if verbose and err:
                print(f"--- {src}\n{err}")
    objs = [os.path.join(BUILD, s + ".o") for s in SOURCES]
    if force or jobs or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    _build_marshal(force, headers)
    with open(stamp, "w") as f:
        f.write(arch)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
