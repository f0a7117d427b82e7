"""Builds libsta.so in-tree with nvcc for sm_103a (no cmake, no torch extension machinery).

Each translation unit is compiled in parallel; the shared library links the CUDA
runtime statically, so it loads wherever the NVIDIA driver is present.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libsta.so")
BIND = os.path.join(HERE, "_bind.so")  # some of the Python calls
SOURCES = ["api.cu", "encode.cu", "mha_row.cu", "mha_block.cu", "decode.cu", "decode_noalloc.cu", "epilogue.cu", "validate.cu", "mla.cu",
           "diag.cu", "rope.cu", "norm_rope.cu", "chunk.cu", "pages.cu"]
HEADERS = ["common.cuh", "internal.h", "ptx.cuh", "rope.inl", "shares.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsta")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                   "-I", os.path.join(ROOT, "include"), "-I", CSRC, *extra]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _bind_commands(obj: str, out: str):
    """g++ commands for csrc/bind.cpp, against the installed torch and libsta.so beside it."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           os.path.join(ROOT, "include")]
    cc = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[f"-I{i}" for i in inc], "-c", os.path.join(CSRC, "bind.cpp"), "-o", obj]
    ld = ["g++", "-shared", "-o", out, obj, f"-L{os.path.join(root, 'lib')}", f"-L{HERE}", "-l:libsta.so", "-lc10", "-lc10_cuda",
          "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    return cc, ld


def _bind_made_for(cc) -> str:
    """What _bind.so was compiled for: its classes are those of this torch's headers, its name's form is this Python's."""
    import sysconfig

    import torch

    return "\n".join([torch.__version__, str(sysconfig.get_config_var("SOABI")), " ".join(cc)])


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "sta.h")]
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        if force or _stale(o, [s] + hdrs):
            jobs.append([nvcc(), *_flags(extra_flags), "-c", s, "-o", o])
    bind_obj, bind_tmp = os.path.join(BUILD, "bind.o"), BIND + f".tmp{os.getpid()}"
    cc, ld = _bind_commands(bind_obj, bind_tmp)
    key_file, key = os.path.join(BUILD, "bind.key"), _bind_made_for(cc)
    made_for = ""
    if os.path.exists(key_file):
        with open(key_file, encoding="utf-8") as f:
            made_for = f.read()
    if force or made_for != key or _stale(bind_obj, [os.path.join(CSRC, "bind.cpp"), os.path.join(ROOT, "include", "sta.h")]):
        jobs.append(cc)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            res = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, res):
            if verbose or r.returncode:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError(f"compilation failed: {' '.join(cmd)}")
    objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of libsta.so failed")
        os.replace(tmp, LIB)
    if force or cc in jobs or _stale(BIND, [bind_obj]):
        r = subprocess.run(ld, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link of _bind.so failed")
        os.replace(bind_tmp, BIND)
        with open(key_file, "w", encoding="utf-8") as f:
            f.write(key)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ())
    print(LIB)
