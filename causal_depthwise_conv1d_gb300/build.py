"""Build libccv.so (the C-ABI CUDA library) in-tree with nvcc for sm_103a.

Every translation unit under ``csrc/`` is compiled in parallel to an object
file in ``_build/`` and linked into ``libccv.so`` next to this file.  The CUDA
runtime is linked as a shared library so the process has one runtime (the
one PyTorch loads) and one notion of the current device.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libccv.so")
EXT_SRC = os.path.join(HERE, "ext", "mixer_ext.cpp")
EXT = os.path.join(HERE, "_mixer_ext.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda_home, "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found (set CUDA_HOME)")
    return found


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _ext_command(out: str):
    """g++ command of the tensor front end (mixer.py), which takes the C ABI from the loaded libccv.so."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    inc = cpp_extension.include_paths() + [INCLUDE, sysconfig.get_paths()["include"],
                                           os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    lib = cpp_extension.library_paths()
    return (["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
            + [f"-isystem{p}" for p in inc] + [EXT_SRC, "-o", out] + [f"-L{p}" for p in lib] +
            [f"-Wl,-rpath,{p}" for p in lib] + ["-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda",
                                                "-Wl,-rpath,$ORIGIN"])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(EXT):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    return all(os.path.getmtime(p) <= t for p in _deps() + [EXT_SRC])


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libccv.so; returns its path.  No-op when up to date."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                     "--expt-relaxed-constexpr"]
    if ptxas_info:
        common += ["-Xptxas", "-v"]
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [nvcc] + common + ["-c", src, "-o", obj]
        if src.endswith(".cpp"):
            cmd = [nvcc] + common + ["-x", "cu", "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    # finished files are moved into place together; nothing else is left if a step fails
    tmp, ext_tmp = (os.path.join(BUILD, f"{os.path.basename(f)}.{os.getpid()}") for f in (LIB, EXT))
    try:
        procs.append((EXT_SRC, subprocess.Popen(_ext_command(ext_tmp), stdout=subprocess.PIPE,
                                                stderr=subprocess.STDOUT)))
        failed = []
        logs = []
        for src, p in procs:
            out, _ = p.communicate()
            text = out.decode(errors="replace")
            if text.strip():
                logs.append(f"== {os.path.basename(src)}\n{text}")
            if p.returncode != 0:
                failed.append(src)
        if failed:
            raise RuntimeError("compilation failed for " + ", ".join(failed) + "\n" + "\n".join(logs))
        if verbose or ptxas_info:
            print("\n".join(logs), file=sys.stderr)
        link = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs
        subprocess.run(link, check=True)
        os.replace(tmp, LIB)
        os.replace(ext_tmp, EXT)
    finally:
        for f in (tmp, ext_tmp):
            if os.path.exists(f):
                os.remove(f)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    info = "--ptxas-info" in sys.argv
    print(build(force=force, verbose="-v" in sys.argv, ptxas_info=info))
