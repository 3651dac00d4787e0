"""Build libarfuse.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel; the shared library links the CUDA
runtime statically so it does not depend on which libcudart the host process
loaded.  Output: ``tp_reduce_moe_gb300/lib/libarfuse.so`` (git-ignored), and
beside it ``_marshal.<torch version>.<Python's ABI>.so``, the binding's native
module (host code, compiled against the headers of the installed torch and of the
interpreter that builds; left out where torch's are missing).
"""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", "arfuse")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libarfuse.so")

SOURCES = ["api.cu", "cluster_rows.cu", "stream_rows.cu", "split_rows.cu", "mhc_post.cu",
           "moe_api.cu", "moe_route.cu", "moe_experts.cu", "matvec_w4.cu",
           "norm_q8.cu", "attn_api.cu", "attn_append.cu", "attn_decode.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libarfuse")


def torch_paths() -> tuple[str, str] | None:
    """torch's folder and version (without importing it); None where it is not installed."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    root = spec.submodule_search_locations[0]
    with open(os.path.join(root, "version.py")) as f:
        version = re.search(r"__version__ = '([^']+)'", f.read()).group(1)
    return root, version


def marshal_path() -> str:
    """Where the native module of this torch and this interpreter lies: neither takes another's."""
    paths = torch_paths()
    return os.path.join(LIBDIR, f"_marshal.{paths[1] if paths else 'none'}.{sysconfig.get_config_var('SOABI')}.so")


def _can_marshal() -> bool:
    paths = torch_paths()
    return (paths is not None and os.path.exists(os.path.join(paths[0], "include", "torch", "csrc", "autograd", "python_variable.h"))
            and os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")))


def _marshal_command(target: str) -> list[str]:
    root, _ = torch_paths()
    return [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
            "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
            "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
            os.path.join(CSRC, "marshal.cpp"), "-o", target, "-L", os.path.join(root, "lib"), "-ltorch_python", "-lc10"]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "arfuse.h"))
    cc = nvcc()
    procs, objs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        objs.append(o)
        if force or ptxas_info or _stale(o, [s] + headers):
            cmd = [cc, *NVCC_FLAGS, "-c", s, "-o", o]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT, text=True)))
    # the native module beside the library, which does without it
    marshal = marshal_path()
    marshal_tmp = marshal + f".tmp{os.getpid()}"
    remade = force or _stale(marshal, [os.path.join(CSRC, "marshal.cpp"), os.path.join(INCLUDE, "arfuse.h")])
    if remade and not _can_marshal():
        print("native module of the binding left out: the headers of torch or Python are missing", file=sys.stderr)
        remade = False
    if remade:
        procs.append(("marshal.cpp", subprocess.Popen(_marshal_command(marshal_tmp), stdout=subprocess.PIPE,
                                                      stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or ptxas_info or p.returncode):
            print(out, file=sys.stderr)
        if p.returncode:
            failed.append(src)
    if any(src != "marshal.cpp" for src in failed):
        raise RuntimeError(f"the compiler failed on {failed}")
    if _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    if failed:
        raise RuntimeError(f"the compiler failed on {failed} (the library is built)")
    if remade:
        os.replace(marshal_tmp, marshal)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
