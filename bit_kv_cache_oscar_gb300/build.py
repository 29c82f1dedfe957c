"""Build liboscar.so in-tree with nvcc for sm_103a (one -gencode, TUs compiled in parallel), and _marshal.so, the
Python-side argument checks of the per-token calls, with g++ against the installed torch."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liboscar.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CUDA_HOME = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def nvcc() -> str:
    p = os.path.join(CUDA_HOME, "bin", "nvcc")
    return p if os.path.exists(p) else (shutil.which("nvcc") or "nvcc")


def sources() -> list:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(out: str, deps: list) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _marshal_flags() -> tuple:
    """(compile, link) flags of the Python extension."""
    import torch
    root = os.path.dirname(torch.__file__)
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    inc = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(CUDA_HOME, "include")]
    libs = os.path.join(root, "lib")
    return (["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={abi}"] + [f"-I{i}" for i in inc],
            [f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{libs}", "-ldl"])


def _stamp(path: str, text: str) -> str:
    """A file that holds `text` and is as old as that."""
    if not os.path.exists(path) or open(path).read() != text:
        with open(path, "w") as f:
            f.write(text)
    return path


def build(verbose: bool = False, extra: list | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    public = [os.path.join(ROOT, "include", f) for f in ("oscar.h", "oscar_int4.h", "oscar_tree.h")]
    headers += public
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                    "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr",
                    "-Xptxas", "-warn-spills"] + (extra or [])
    objs, procs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if _stale(obj, [src, *headers]):
            cmd = [nvcc(), *flags, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    msrc, mobj = os.path.join(CSRC, "marshal.cpp"), os.path.join(BUILD, "marshal.o")
    mflags = _marshal_flags()
    import torch
    made_with = _stamp(os.path.join(BUILD, "marshal.made_with"), repr((mflags, torch.__version__, sys.version)))
    if _stale(mobj, [msrc, made_with, *public]):
        cmd = ["g++", *mflags[0], "-c", msrc, "-o", mobj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((msrc, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(text, flush=True)
    if failed:
        for src, text in failed:
            sys.stderr.write(f"compiling {src} failed:\n{text}\n")
        raise RuntimeError("liboscar.so build failed")
    if _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
               "-Xlinker", f"-rpath,{os.path.join(CUDA_HOME, 'lib64')}"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    if _stale(MARSHAL, [mobj]):
        tmp = MARSHAL + f".tmp{os.getpid()}"
        cmd = ["g++", "-shared", "-o", tmp, mobj, *mflags[1]]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, MARSHAL)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
