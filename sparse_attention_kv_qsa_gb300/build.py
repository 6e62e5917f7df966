"""Builds ``libqsa.so`` (the C ABI of include/qsa.h) for sm_103a with nvcc, and
``qsa_ops.so``, the Python module that binds the bounded-cache calls to torch.

Each CUDA source compiles to an object in parallel (the module's one C++ source
beside them), then one link step makes the shared library in ``_build/`` and
another the module, which links to it. The CUDA runtime is linked statically
into ``libqsa.so``, so the library needs only the driver at run time; the module
needs the torch that it was built against.
"""

from __future__ import annotations

import concurrent.futures
import hashlib
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libqsa.so")
INCLUDE = os.path.join(ROOT, "include")
BINDING = os.path.join(HERE, "binding", "qsa_ops.cpp")
OPS = os.path.join(BUILD, "qsa_ops.so")
OPS_KEY = OPS + ".key"   # what the module was linked against: binding_key()

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqsa.so")
    return path


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers_mtime() -> float:
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(INCLUDE, "qsa.h"))
    return max(os.path.getmtime(h) for h in hs)


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), _headers_mtime()) \
            and not extra:
        return obj
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def binding_key() -> str:
    """The torch and the Python that a built module belongs to: it uses both their C++ and C interfaces."""
    import torch
    return f"torch {torch.__version__} {_torch_dir()}, {sysconfig.get_config_var('SOABI')}"


def linked_for() -> str | None:
    """The ``binding_key()`` that ``qsa_ops.so`` was linked for; None where there is no module, or it does not say."""
    if not os.path.exists(OPS) or not os.path.exists(OPS_KEY):
        return None
    with open(OPS_KEY) as f:
        return f.read()


def _compile_binding(force: bool) -> str:
    """The module's object; one for each binding_key(), rebuilt when its source or the header changed."""
    import torch
    obj = os.path.join(BUILD, f"qsa_ops.{hashlib.sha256(binding_key().encode()).hexdigest()[:16]}.obj")
    newest = max(os.path.getmtime(BINDING), os.path.getmtime(os.path.join(INCLUDE, "qsa.h")))
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj
    t = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", t,
           "-I", os.path.join(t, "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"], "-I", cuda,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-c", BINDING, "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj


def _binding_is_current(obj: str) -> bool:
    # By the key and not by times alone: another torch's object may be the older one and yet not the one linked.
    return linked_for() == binding_key() and os.path.getmtime(OPS) >= max(os.path.getmtime(obj), os.path.getmtime(LIB))


def _link_binding(obj: str) -> None:
    lib = os.path.join(_torch_dir(), "lib")
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", OPS + ".tmp", obj, "-L", BUILD, "-l:libqsa.so", "-L", lib,
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {OPS} failed:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(OPS_KEY):
        os.remove(OPS_KEY)   # a module without a key is linked again
    os.replace(OPS + ".tmp", OPS)
    with open(OPS_KEY + ".tmp", "w") as f:
        f.write(binding_key())
    os.replace(OPS_KEY + ".tmp", OPS_KEY)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every CUDA source and link libqsa.so, then qsa_ops.so; returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    if force:
        for f in os.listdir(BUILD):
            if f.endswith(".o"):
                os.remove(os.path.join(BUILD, f))
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=1 + min(8, len(srcs))) as ex:
        binding = ex.submit(_compile_binding, force)
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
        ops = binding.result()
    if force or extra or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [nvcc(), *ARCH, "-shared", "-o", LIB + ".tmp", *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(LIB + ".tmp", LIB)
    if force or not _binding_is_current(ops):
        _link_binding(ops)
    return LIB


if __name__ == "__main__":
    print(build(force=True))
