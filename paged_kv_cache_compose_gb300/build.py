"""Build ``libcpkv.so`` in-tree with nvcc for sm_103a, and ``_serving``, the
Python marshalling of the serving calls, with the host compiler against the
torch that is installed (left out where there is none: the library and the
compose need neither).

Each translation unit under ``csrc/`` is compiled in parallel, then linked
into one shared library next to this file.  Usage::

    python -m paged_kv_cache_compose_gb300.build          # build if stale
    python -m paged_kv_cache_compose_gb300.build --force  # rebuild
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libcpkv.so")
BINDING_SRC = os.path.join(CSRC, "serving_binding.cpp")
BINDING_PATH = os.path.join(HERE, "_serving" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_STAMP = os.path.join(BUILD_DIR, "serving_binding.torch")  # version of torch that it was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


_ELF_MACHINE = {"x86_64": 62, "aarch64": 183}  # ELF e_machine of this host's shared objects


def _built_for_other_machine(path: str) -> bool:
    """True when ``path`` is an ELF object for another CPU than this host's
    (a library copied over from a machine of another architecture)."""
    import platform

    want = _ELF_MACHINE.get(platform.machine())
    try:
        with open(path, "rb") as f:
            head = f.read(20)
    except OSError:
        return True
    if want is None or len(head) < 20 or head[:4] != b"\x7fELF":
        return want is not None
    return int.from_bytes(head[18:20], "little") != want


def _older(path: str, deps: list[str]) -> bool:
    if not os.path.exists(path) or _built_for_other_machine(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in deps)


def stale() -> bool:
    return _older(LIB_PATH, _deps())


def torch_version() -> str | None:
    """Of the installed torch, without importing it; None where there is none."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


def binding_stale() -> bool:
    version = torch_version()
    if version is None:
        return False
    try:
        with open(BINDING_STAMP) as f:
            built_for = f.read()
    except OSError:
        return True
    return built_for != version or _older(BINDING_PATH, [BINDING_SRC, os.path.join(INCLUDE, "cpkv.h")])


def _torch_dirs() -> tuple[list[str], str]:
    """torch's include directories and its library directory."""
    import torch

    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    return [inc, os.path.join(inc, "torch", "csrc", "api", "include")], os.path.join(root, "lib")


def _compile_binding() -> str:
    import torch

    obj = os.path.join(BUILD_DIR, "serving_binding.o")
    inc = [INCLUDE, *_torch_dirs()[0], sysconfig.get_paths()["include"]]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DBUILT_FOR="{torch_version()}"',
           *[a for d in inc for a in ("-isystem" if "torch" in d else "-I", d)], "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(BINDING_SRC)}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    lib = _torch_dirs()[1]
    tmp = BINDING_PATH + f".{os.getpid()}.tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", HERE, "-lcpkv", "-L", lib, "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(BINDING_PATH)} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w") as f:
        f.write(torch_version())


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every CUDA translation unit and link ``libcpkv.so``; compile and
    link ``_serving`` beside it."""
    library, binding = force or stale(), binding_stale() or force and torch_version() is not None
    if not library and not binding:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    srcs = sources() if library else []
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        objs = [ex.submit(_compile, s, extra) for s in srcs]
        binding_obj = ex.submit(_compile_binding) if binding else None
        objs = [f.result() for f in objs]
        if library:
            tmp = LIB_PATH + f".{os.getpid()}.tmp"
            cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB_PATH)
        if binding_obj is not None:
            _link_binding(binding_obj.result())
    return LIB_PATH


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print register / shared-memory usage")
    a = ap.parse_args(argv)
    print(build(force=a.force or a.ptxas_v, verbose_ptxas=a.ptxas_v))
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
