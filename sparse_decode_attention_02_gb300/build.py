"""Builds, in-tree, libsdattn.so (the C-ABI library; nvcc for sm_103a) and _marshal.so
(the binding's native argument marshalling; g++ against the installed torch)."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", name) for name in (
    "sdattn.cu", "sda_select.cu", "sda_index.cu", "sda_plan.cu", "sda_rope.cu", "sda_quant.cu",
    "sda_paged.cu",
    *(f"sda_paged_{kind}_{dim}.cu" for kind in ("bf16", "fp8", "qe4m3", "qint8") for dim in (64, 128, 192, 256)))]
INCLUDES = [os.path.join(HERE, "csrc", name) for name in ("sda_common.cuh", "sda_context.cuh", "sda_quant.cuh",
                                                           "sda_paged.cuh")]
HEADER = os.path.join(ROOT, "include", "sdattn.h")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libsdattn.so")
MARSHAL_SOURCE = os.path.join(HERE, "csrc", "sda_marshal.cpp")
MARSHAL = os.path.join(OUT_DIR, "_marshal.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None,
          out: str = LIB) -> str:
    """Compile the library unless it is newer than its sources; returns its path."""
    if (not force and not extra and os.path.exists(out)
            and os.path.getmtime(out) >= max(os.path.getmtime(x) for x in [*SOURCES, *INCLUDES, HEADER])):
        return out
    os.makedirs(os.path.dirname(out), exist_ok=True)
    tmp = out + f".tmp{os.getpid()}"
    common = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I", os.path.join(ROOT, "include"), *(extra or [])]
    if verbose:
        common.insert(1, "-Xptxas=-v")
    objs = [f"{tmp}.{i}.o" for i in range(len(SOURCES))]
    procs = [subprocess.Popen([*common, "-c", src, "-o", obj], stdout=subprocess.PIPE,
                              stderr=subprocess.PIPE, text=True)
             for src, obj in zip(SOURCES, objs)]            # translation units in parallel
    logs = [p.communicate() for p in procs]
    failed = [p.returncode for p in procs if p.returncode]
    if not failed:
        r = subprocess.run([nvcc(), *ARCH, "-shared", *objs, "-o", tmp], capture_output=True, text=True)
        logs.append((r.stdout, r.stderr))
        failed = [r.returncode] if r.returncode else []
    for obj in objs:
        if os.path.exists(obj):
            os.remove(obj)
    if failed or verbose:
        sys.stderr.write("".join(a + b for a, b in logs))
    if failed:
        raise RuntimeError("nvcc failed building libsdattn.so")
    os.replace(tmp, out)
    return out


def build_marshal(force: bool = False, out: str = MARSHAL) -> str:
    """Compile the marshalling module unless it is newer than its sources; returns its path."""
    import sysconfig

    import torch

    if not force and os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(x)
                                                                           for x in (MARSHAL_SOURCE, HEADER)):
        return out
    os.makedirs(os.path.dirname(out), exist_ok=True)
    base = os.path.dirname(torch.__file__)
    lib = os.path.join(base, "lib")
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = out + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", MARSHAL_SOURCE, "-o", tmp,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
           *(a for d in (os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
                         os.path.join(cuda, "include")) for a in ("-isystem", d)),
           "-L", lib, f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]   # libcudart: c10_cuda's
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("g++ failed building _marshal.so")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
    build_marshal(force=True)
    print(LIB)
