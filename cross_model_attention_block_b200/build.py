"""Build libmapflow.so in-tree for sm_100a (nvcc + g++; no GPU needed).

    python -m cross_model_attention_block_b200.build [--force] [--jobs N]

Objects go to cross_model_attention_block_b200/_build/, the library to
cross_model_attention_block_b200/libmapflow.so.  A source is recompiled when it
or any header is newer than its object.  The argument marshalling of the decode
calls (csrc_py/, against torch's headers) becomes _marshal.so beside it, again
whenever torch or Python are others than it was built for.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmapflow.so")
MARSHAL_SRC = os.path.join(PKG, "csrc_py", "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_FOR = os.path.join(PKG, "_build", "marshal_for")  # marshal_key() of the built one
CUDA_HOME = os.environ.get("CUDA_HOME", "/usr/local/cuda")
NVCC = os.path.join(CUDA_HOME, "bin", "nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
              "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]
CXX_FLAGS = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-I" + os.path.join(ROOT, "include")]


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(src, obj, hdr_mtime):
    if not os.path.exists(obj):
        return True
    m = os.path.getmtime(obj)
    return os.path.getmtime(src) > m or hdr_mtime > m


def _compile(src, obj, verbose_ptxas=False):
    if src.endswith(".cu"):
        cmd = [NVCC] + ARCH + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose_ptxas else []) + \
              ["-c", src, "-o", obj]
    else:
        cmd = ["g++"] + CXX_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stderr


def marshal_key() -> str:
    """What _marshal.so's inlined accesses to torch's and Python's objects depend on."""
    import sysconfig

    import torch
    return (f"torch {torch.__version__} abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} "
            f"{sysconfig.get_config_var('SOABI')}")


def _marshal_stale(key: str) -> bool:
    hdr = os.path.join(ROOT, "include", "mapflow.h")
    if _stale(MARSHAL_SRC, MARSHAL, os.path.getmtime(hdr)) or not os.path.exists(MARSHAL_FOR):
        return True
    with open(MARSHAL_FOR) as f:
        return f.read() != key


def build_marshal(force: bool = False) -> str:
    """Compile _marshal.so against the running interpreter's torch."""
    key = marshal_key()
    if not force and not _marshal_stale(key):
        return MARSHAL
    import sysconfig

    import torch
    troot = os.path.dirname(torch.__file__)
    inc = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"],
           os.path.join(CUDA_HOME, "include"), os.path.join(troot, "include"),
           os.path.join(troot, "include", "torch", "csrc", "api", "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DMF_MARSHAL_KEY="{key}"']
    for i in inc:
        cmd += ["-isystem" if troot in i else "-I", i]
    tmp = MARSHAL + ".tmp"
    cmd += [MARSHAL_SRC, "-o", tmp, "-L" + os.path.join(troot, "lib"), "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    shutil.move(tmp, MARSHAL)
    os.makedirs(os.path.dirname(MARSHAL_FOR), exist_ok=True)
    with open(MARSHAL_FOR, "w") as f:
        f.write(key)
    return MARSHAL


def build(force: bool = False, jobs: int = 8, verbose_ptxas: bool = False) -> str:
    """Compile every kernel source for sm_100a and link libmapflow.so."""
    if not os.path.exists(NVCC):
        raise RuntimeError(f"nvcc not found at {NVCC}")
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))
    hdr = max([os.path.getmtime(h) for h in _headers()] + [0.0])
    objs, todo = [], []
    for s in srcs:
        o = os.path.join(OUT_DIR, os.path.basename(s) + ".o")
        objs.append(o)
        if force or _stale(s, o, hdr):
            todo.append((s, o))
    logs = []
    if todo:
        with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
            for log in ex.map(lambda so: _compile(so[0], so[1], verbose_ptxas), todo):
                if log:
                    logs.append(log)
    if todo or not os.path.exists(LIB):
        tmp = LIB + ".tmp"
        cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            # the driver library may only exist as a stub on a build host
            cmd = cmd[:-1] + ["-L" + os.path.join(CUDA_HOME, "lib64", "stubs"), "-lcuda"]
            r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        shutil.move(tmp, LIB)
    if verbose_ptxas:
        print("\n".join(logs))
    build_marshal(force)
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--jobs", type=int, default=8)
    ap.add_argument("--ptxas", action="store_true", help="print -Xptxas -v output")
    a = ap.parse_args()
    print(build(a.force, a.jobs, a.ptxas))


if __name__ == "__main__":
    sys.exit(main())
