"""Build libkda (the CUDA path) in-tree with nvcc for sm_103a.

Translation units are compiled in parallel and linked into
``kda_linear_attention_bounded_gb300/_build/libkda.so``.  ``csrc/kda_torch.cpp``
(torch tensors' argument checks) becomes a module beside it, named after the
interpreter and the torch it is for (:func:`torch_ext`); the library is built and
linked without it, too (``build(binding=False)``, ``--library``), and is in place
whatever becomes of the module.  The CUDA runtime is linked statically and the
driver API (tensor-map encoding) is resolved at run time, so the library loads on
a machine without a GPU driver.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libkda.so")
TORCH_SRC = os.path.join(CSRC, "kda_torch.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def torch_ext() -> str:
    """The module's path for the running interpreter and torch (another one's is never loaded)."""
    import torch

    return os.path.join(BUILD, f"_kda_torch.{sys.implementation.cache_tag}-torch{torch.__version__}.so")


def _fresh(target, deps):
    return os.path.exists(target) and os.path.getmtime(target) >= max(os.path.getmtime(p) for p in deps)


def _library_deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(INCLUDE, "kda.h"), os.path.abspath(__file__)]


def _binding_deps():
    return [TORCH_SRC, os.path.join(INCLUDE, "kda.h"), os.path.abspath(__file__)]


def _torch_ext_command(out):
    import sysconfig

    import torch

    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}", f"-I{root}/include",
            f"-I{root}/include/torch/csrc/api/include", f"-I{cuda}/include", f"-I{sysconfig.get_paths()['include']}",
            TORCH_SRC, "-o", out, f"-L{root}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    except OSError as e:   # (no such compiler)
        return e


def _finish(started, verbose):
    """What failed of (source, process) pairs, with its output."""
    failed = []
    for src, p in started:
        if isinstance(p, OSError):
            failed.append(f"{src}:\n{p}")
            continue
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append(f"{src}:\n{out}")
        elif verbose and out:
            print(out, file=sys.stderr)
    return failed


def build(force: bool = False, verbose: bool = False, extra_flags=(), binding: bool = True) -> str:
    """Build what is not up to date: the library, and the torch binding's module unless ``binding`` is false."""
    os.makedirs(BUILD, exist_ok=True)
    need_lib = force or not _fresh(LIB, _library_deps())
    ext = torch_ext() if binding else None
    need_ext = binding and (force or not _fresh(ext, _binding_deps()))
    units, objs, module = [], [], []
    if need_lib:
        for src in sources():
            obj = os.path.join(BUILD, os.path.basename(src) + ".o")
            units.append((src, _start([_nvcc(), *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj], verbose)))
            objs.append(obj)
    ext_tmp = f"{ext}.tmp{os.getpid()}"
    if need_ext:
        module.append((TORCH_SRC, _start(_torch_ext_command(ext_tmp), verbose)))
    failed, module_failed = _finish(units, verbose), _finish(module, verbose)
    if need_lib and not failed:
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([_nvcc(), *ARCH, "-shared", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    if need_ext and not module_failed:
        os.replace(ext_tmp, ext)
    if failed or module_failed:
        raise RuntimeError("compilation failed:\n" + "\n".join(failed + module_failed))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, binding="--library" not in sys.argv))
