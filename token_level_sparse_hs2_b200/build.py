"""Builds libhs2.so (the CUDA kernels + C ABI) in-tree for sm_100a with nvcc, and the Python module
_marshal.so (csrc/marshal.cpp: torch tensors to C ABI calls) against it with the host compiler. The
library needs nvcc alone: it is linked whether or not the module can be made, and without torch the module is left out.

Usage: python -m token_level_sparse_hs2_b200.build [--force]
Object files go to token_level_sparse_hs2_b200/_build/; the library to
token_level_sparse_hs2_b200/libhs2.so, the module beside it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libhs2.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found")
    return exe


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  [os.path.join(ROOT, "include", "hs2.h")])


def _compile(src: str, obj: str, verbose: bool) -> str:
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stderr}")
    return res.stderr


def _marshal_stamp():
    """What marshal.cpp.o depends on besides its sources: the torch and the Python it is compiled against. None
    without torch."""
    try:
        import torch
    except ImportError:
        return None
    return "\n".join([torch.__version__, os.path.dirname(torch.__file__), str(torch._C._GLIBCXX_USE_CXX11_ABI),
                      str(sysconfig.get_config_var("EXT_SUFFIX")), sysconfig.get_paths()["include"]])


def _marshal_object(src: str, obj: str) -> None:
    """Compiles marshal.cpp against torch's headers."""
    import torch
    inc = [os.path.join(os.path.dirname(torch.__file__), "include"), sysconfig.get_paths()["include"],
           os.path.join(ROOT, "include")]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", *["-I" + i for i in inc],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{res.stderr}")


def _marshal_link(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L" + HERE, "-l:libhs2.so", "-L" + lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, MARSHAL)


def _link(objs) -> None:
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIB)


def _older(path: str, than) -> bool:
    """Whether `path` is missing or older than one of the files."""
    return not os.path.exists(path) or os.path.getmtime(path) < max(os.path.getmtime(p) for p in than)


def _read(path: str):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    dep_mtime = max(os.path.getmtime(p) for p in _deps())
    jobs = []
    objs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or \
                os.path.getmtime(obj) < max(os.path.getmtime(src), dep_mtime):
            jobs.append((src, obj))
    # The module is made anew when its sources, torch or Python have changed, and linked anew whenever it is older
    # than its object (an earlier call may have failed in between): after a change of hs2.h an older one would
    # call the library with the arguments of before.
    msrc, mobj = os.path.join(CSRC, "marshal.cpp"), os.path.join(BUILD, "marshal.cpp.o")
    mdeps = [msrc, os.path.join(ROOT, "include", "hs2.h")]
    mstamp, stamp = os.path.join(BUILD, "marshal.stamp"), _marshal_stamp()
    m_job = stamp is not None and (force or _older(mobj, mdeps) or _read(mstamp) != stamp)
    try:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(jobs) + 1)) as ex:
            marshal = ex.submit(_marshal_object, msrc, mobj) if m_job else None
            logs = list(ex.map(lambda j: _compile(j[0], j[1], verbose), jobs))
        if verbose:
            for log in logs:
                sys.stderr.write(log)
        if force or _older(LIB, objs):
            _link(objs)
        if marshal is not None:
            marshal.result()
            with open(mstamp, "w") as f:
                f.write(stamp)
        if stamp is None:
            sys.stderr.write("torch cannot be imported: libhs2.so is built, the Python module _marshal.so is not\n")
            if os.path.exists(MARSHAL) and _older(MARSHAL, mdeps):
                os.remove(MARSHAL)
        elif force or _older(MARSHAL, [mobj]):
            _marshal_link(mobj)
    except BaseException:
        # no module that does not match what is (or the next call finds) built
        if os.path.exists(MARSHAL) and (m_job or _older(MARSHAL, mdeps)):
            os.remove(MARSHAL)
        raise
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
