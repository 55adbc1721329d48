"""Builds librmsnorm.so in-tree from csrc/*.cu for sm_103a (GB300).

Each translation unit is compiled by its own nvcc process (in parallel), then
linked into ``_build/librmsnorm.so`` against the shared CUDA runtime, so the
library and PyTorch share one runtime state. A rebuild happens only when a
source or header is newer than the library.

A second, checked variant of the same sources (``-DRMSNORM_CHECKS``, in
``_build_checked/``) tests every global store, bulk copy and shared-memory
ring access of the kernels against the extent it belongs to and reports a
failed check as RMSNORM_ERR_OUT_OF_BOUNDS instead of making the access. It is
a debug build for the tests; the binding loads it only when
RMSNORM_LIBRARY_VARIANT=checked is set.

The Python binding of the tensor-level image operators (csrc/binding.cpp, host
code only, compiled by g++ against PyTorch's headers) goes to
``_build/_binding.so`` and serves both variants; without a PyTorch that has CUDA it
is left out. It is compiled again when PyTorch or Python is another version than the
one it was made for.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
CHECKED_BUILD_DIR = os.path.join(PKG_DIR, "_build_checked")
LIB_NAME = "librmsnorm.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
CHECKED_LIB_PATH = os.path.join(CHECKED_BUILD_DIR, LIB_NAME)
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(BUILD_DIR, "_binding.so")

SOURCES = ["api.cu", "fwd.cu", "bwd.cu", "bwd_f32.cu", "bwd_bf16.cu", "bwd_f16.cu",
           "bwd_res_f32.cu", "bwd_res_bf16.cu", "bwd_res_f16.cu", "naive.cu", "probe.cu",
           "noalloc.cu", "rope.cu", "rope_f32.cu", "rope_bf16.cu", "rope_f16.cu",
           "pair_sum.cu", "group_norm.cu",
           "group_norm_f32.cu", "group_norm_bf16.cu", "group_norm_f16.cu", "group_norm_scalar.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build librmsnorm.so")


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
             if f.endswith((".cu", ".cuh", ".h"))]
    files.append(os.path.join(INCLUDE, "rmsnorm.h"))
    files.append(os.path.abspath(__file__))
    return files


def source_hash() -> str:
    """sha256 over the sources the library is built from (for run records)."""
    h = hashlib.sha256()
    for f in _inputs():
        h.update(os.path.basename(f).encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()[:16]


BWD_KERNEL_FILES = ("bwd.cu", "bwd_kernels.cuh", "bwd_f32.cu", "bwd_bf16.cu", "bwd_f16.cu",
                    "bwd_res_f32.cu", "bwd_res_bf16.cu", "bwd_res_f16.cu", "common.cuh",
                    "kernels.h")


FWD_KERNEL_FILES = ("fwd.cu", "common.cuh", "kernels.h")


def kernel_source_hash(names=BWD_KERNEL_FILES) -> str:
    """sha256 over the csrc files that define a kernel family (by default the
    backward), so a profile can be matched to the kernel code it measured."""
    h = hashlib.sha256()
    for n in names:
        h.update(n.encode())
        with open(os.path.join(CSRC, n), "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()[:16]


def lib_path(checked: bool = False) -> str:
    return CHECKED_LIB_PATH if checked else LIB_PATH


def is_stale(checked: bool = False) -> bool:
    path = lib_path(checked)
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _torch_dir() -> str | None:
    """Where PyTorch lies, None without one that has CUDA."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    path = list(spec.submodule_search_locations)[0]
    return path if os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def _binding_made_for() -> str:
    """The versions whose interfaces the binding is compiled against."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "of unknown version"
    return f"torch {torch} in {_torch_dir()}, {sys.implementation.cache_tag}"


def binding_is_stale() -> bool:
    if _torch_dir() is None:
        return False
    if not os.path.exists(BINDING_PATH):
        return True
    try:
        with open(BINDING_PATH + ".info") as fh:
            if fh.read() != _binding_made_for():
                return True
    except OSError:
        return True
    t = os.path.getmtime(BINDING_PATH)
    return any(os.path.getmtime(f) > t for f in
               (BINDING_SOURCE, os.path.join(INCLUDE, "rmsnorm.h"), os.path.abspath(__file__)))


def _build_binding() -> None:
    torch = _torch_dir()
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    includes = [INCLUDE, os.path.join(torch, "include"),
                os.path.join(torch, "include", "torch", "csrc", "api", "include"), cuda,
                sysconfig.get_paths()["include"]]
    os.makedirs(BUILD_DIR, exist_ok=True)
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    _run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
          *(f"-I{d}" for d in includes), BINDING_SOURCE, "-o", tmp,
          "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
          "-ltorch", "-ltorch_python"], os.path.join(BUILD_DIR, "binding.log"))
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_PATH + ".info", "w") as fh:
        fh.write(_binding_made_for())


def _run(cmd: list[str], log: str | None) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    out = (res.stdout or "") + (res.stderr or "")
    if log:
        with open(log, "w") as fh:
            fh.write(" ".join(cmd) + "\n" + out)
    if res.returncode != 0:
        raise RuntimeError(f"command failed ({res.returncode}): {' '.join(cmd)}\n{out}")


def _variant_jobs(checked: bool, extra: list[str]):
    """(compile commands, objects, link step) of one variant."""
    nvcc = _nvcc()
    out_dir = CHECKED_BUILD_DIR if checked else BUILD_DIR
    os.makedirs(out_dir, exist_ok=True)
    defs = ["-DRMSNORM_CHECKS"] if checked else []
    objs, cmds = [], []
    for src in SOURCES:
        obj = os.path.join(out_dir, src.replace(".cu", ".o"))
        objs.append(obj)
        log = os.path.join(out_dir, src.replace(".cu", ".log"))
        cmds.append(([nvcc, *ARCH, *FLAGS, *defs, *extra, "-c", os.path.join(CSRC, src), "-o",
                      obj], log))
    return cmds, objs, out_dir


def _link(objs: list[str], checked: bool) -> None:
    path = lib_path(checked)
    tmp = path + f".tmp{os.getpid()}"
    _run([_nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs], None)
    os.replace(tmp, path)
    with open(os.path.join(os.path.dirname(path), "BUILD_INFO"), "w") as fh:
        fh.write(f"source_hash={source_hash()}\nnvcc={_nvcc()}\narch=sm_103a\n"
                 f"checked={int(checked)}\n")


def build(force: bool = False, ptxas_verbose: bool = False, jobs: int | None = None,
          checked: bool = False, both: bool = False) -> str:
    """Compile and link the library if needed; returns its path. `checked`
    builds the checked debug variant instead; `both` builds the library and
    the checked variant together (one pool of compile jobs) and returns the
    library's path."""
    variants = [False, True] if both else [checked]
    todo = [v for v in variants if force or is_stale(v)]
    binding = _torch_dir() is not None and (force or binding_is_stale())
    if not todo and not binding:
        return lib_path(checked and not both)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    plans = {v: _variant_jobs(v, extra) for v in todo}
    cmds = [c for v in todo for c in plans[v][0]]
    workers = jobs or min(len(cmds) + 1, max(1, os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(max_workers=workers) as ex:
        of_binding = ex.submit(_build_binding) if binding else None
        futures = [ex.submit(_run, c, log) for c, log in cmds]
        for fut in futures:
            fut.result()
    for v in todo:
        _link(plans[v][1], v)
    if of_binding is not None:
        of_binding.result()  # the library does not depend on it
    return lib_path(checked and not both)


if __name__ == "__main__":
    path = build(force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv,
                 checked="--checked" in sys.argv, both="--both" in sys.argv)
    print(path)
