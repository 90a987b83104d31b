"""Builds libtefwd.so in the package directory with nvcc for sm_103a, and the
binding's marshalling module next to it.

Each CUDA translation unit compiles in parallel to an object under _build/,
then one nvcc link produces the shared library (CUDA runtime linked
statically).  The marshalling module (csrc/marshal.cpp: a CPython extension
over PyTorch's headers) compiles beside them where PyTorch is installed.  Run
``python -m transformer_encoder_forward_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtefwd.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
SOURCES = ["rowops.cu", "q8_linear.cu", "attn.cu", "block.cu", "block_static.cu", "codecs.cu",
           "quant.cu", "i8_linear.cu", "rope_axes.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _have_torch() -> bool:
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def _marshal_flags():
    """Compile and link flags of the marshalling module (PyTorch's and Python's)."""
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    comp = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
            "-isystem", os.path.join(root, "include"),
            "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"]]
    libs = os.path.join(root, "lib")
    link = ["-L", libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{libs}"]
    return comp, link


def _marshal_key(cxx, comp, link) -> str:
    import torch
    return "\n".join([torch.__version__, str(torch.version.git_version), sys.version, cxx, *comp, *link])


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except FileNotFoundError:
        return ""


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    cc = nvcc()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s, *headers]):
            jobs.append([cc, *ARCH, *FLAGS, *extra, "-c", s, "-o", o])
    cuda_jobs = len(jobs)
    # The library needs no PyTorch; where there is none, neither does anybody
    # call the module.
    with_module = _have_torch()
    if with_module:
        comp, link = _marshal_flags()
        cxx = os.environ.get("CXX") or "g++"
        m_src, m_obj = os.path.join(CSRC, "marshal.cpp"), os.path.join(BUILD, "marshal.o")
        # what the module's object and binary were made for: another PyTorch or
        # Python, which neither file's time shows, makes them anew
        m_key, key = os.path.join(BUILD, "marshal.key"), _marshal_key(cxx, comp, link)
        m_new = force or _read(m_key) != key
        if m_new or _stale(m_obj, [m_src, os.path.join(INCLUDE, "tefwd.h")]):
            jobs.append([cxx, *comp, "-c", m_src, "-o", m_obj])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)

    with cf.ThreadPoolExecutor(max_workers=len(jobs) or 1) as ex:
        list(ex.map(run, jobs))
    if force or cuda_jobs or _stale(LIB, objs):
        run([cc, *ARCH, "-shared", "-o", LIB + ".tmp", *objs])
        os.replace(LIB + ".tmp", LIB)
    if with_module and (m_new or _stale(MARSHAL, [m_obj])):
        run([cxx, "-shared", "-o", MARSHAL + ".tmp", m_obj, *link])
        os.replace(MARSHAL + ".tmp", MARSHAL)
        with open(m_key, "w") as f:
            f.write(key)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
