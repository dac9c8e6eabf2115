"""Build the CUDA library in-tree: sparse_attention_indexer_sm_gb300/_build/libtopk_transform.so.

Every object is compiled for sm_103a only, all of them in parallel, then linked
against the shared CUDA runtime (so that the process keeps a single runtime
together with PyTorch). Beside it stands the indexer operators' Python binding, a
C++ module for this interpreter and this PyTorch, linked against the library, which
does not depend on it: a binding that cannot be built leaves the library in place.
Run ``python -m sparse_attention_indexer_sm_gb300.build``.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libtopk_transform.so")

SOURCES = ("topk_select.cu", "topk_api.cu", "indexer_rotary.cu", "indexer_cache.cu",
           "indexer_scores.cu")
# The kernel source is compiled once per (CTA size, form) and once per CTA size for
# the dispatch by form: ten objects that build in parallel.
KERNEL_OBJECTS = [(f"topk_select_{cta}_{form}", ["-DTOPK_CTA_THREADS=%d" % cta, "-DTOPK_FORM=%d" % form])
                  for cta in (512, 256) for form in range(4)]
KERNEL_OBJECTS += [(f"topk_select_{cta}", ["-DTOPK_CTA_THREADS=%d" % cta]) for cta in (512, 256)]
HEADERS = (os.path.join(CSRC, "topk_select.cuh"), os.path.join(CSRC, "indexer_common.cuh"),
           os.path.join(INCLUDE, "topk_transform.h"), os.path.join(INCLUDE, "indexer_ops.h"))
BINDING_SOURCE = os.path.join(CSRC, "indexer_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _pytorch() -> bool:
    """Whether there is a PyTorch to build the binding for."""
    return importlib.util.find_spec("torch") is not None


def binding_path() -> str:
    """The binding's module, of this interpreter's and this PyTorch's version."""
    import torch
    return os.path.join(BUILD_DIR, f"indexer_binding-{sys.implementation.cache_tag}-{torch.__version__}.so")


def _stale() -> bool:
    outs = [LIB_PATH, binding_path()] if _pytorch() else [LIB_PATH]
    if not all(os.path.exists(p) for p in outs):
        return True
    t = min(os.path.getmtime(p) for p in outs)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + list(HEADERS) + [BINDING_SOURCE, __file__]
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_commands(obj: str, out: str, cuda_home: str) -> tuple[list[str], list[str]]:
    """The host compiler's commands for the binding: compile, link."""
    import torch
    base = os.path.dirname(torch.__file__)
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", BINDING_SOURCE, "-o", obj,
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
                "-isystem", os.path.join(base, "include"),
                "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
                "-isystem", os.path.join(cuda_home, "include"),
                "-isystem", sysconfig.get_paths()["include"], "-I" + INCLUDE]
    link = [cxx, "-shared", "-o", out, obj, "-L" + os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch",
            "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-L" + BUILD_DIR, "-ltopk_transform",
            "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed ({' '.join(cmd)}):\n{r.stdout}")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link if any source is newer than the library; return its path."""
    if not force and not _stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    exe = nvcc()
    cuda_home = os.path.dirname(os.path.dirname(os.path.realpath(exe)))
    procs, objs = [], []
    units = [(name, defs, "topk_select.cu") for name, defs in KERNEL_OBJECTS]
    units += [(os.path.splitext(src)[0], [], src) for src in SOURCES[1:]]

    def start(cmd):
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))

    for name, defs, src in units:
        obj = os.path.join(BUILD_DIR, name + ".o")
        cmd = [exe, *NVCC_FLAGS, *defs, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        start(cmd)
        objs.append(obj)
    without_compiler = None
    if _pytorch():
        binding = binding_path()
        binding_tmp = binding + f".{os.getpid()}.tmp"
        compile_binding, link_binding = _binding_commands(os.path.join(BUILD_DIR, "indexer_binding.o"), binding_tmp,
                                                          cuda_home)
        try:
            start(compile_binding)
        except OSError as e:  # raised again once the library stands
            without_compiler = e

    def finish(cmd, p):
        out, _ = p.communicate()
        if p.returncode != 0:
            raise RuntimeError(f"compiler failed ({' '.join(cmd)}):\n{out}")
        if verbose and out:
            print(out, file=sys.stderr)

    for cmd, p in procs[:len(objs)]:
        finish(cmd, p)
    tmp = LIB_PATH + f".{os.getpid()}.tmp"
    cuda_lib = os.path.join(cuda_home, "lib64")
    _run([exe, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-rpath," + cuda_lib,
          "-Xlinker", "-soname,libtopk_transform.so", "-o", tmp, *objs], "link")
    os.replace(tmp, LIB_PATH)
    if without_compiler is not None:
        raise RuntimeError(f"compiler failed ({' '.join(compile_binding)}): {without_compiler}")
    if _pytorch():
        finish(*procs[-1])
        _run(link_binding, "link of the binding")
        os.replace(binding_tmp, binding)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
