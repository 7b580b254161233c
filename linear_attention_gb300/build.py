"""Builds the CUDA library in-tree with nvcc (sm_103a only), and the operators' Python binding with g++."""
from __future__ import annotations

import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB_DIR = os.path.join(HERE, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libbased_gb300.so")
SOURCES = [os.path.join(CSRC, f) for f in ("based_fwd.cu", "based_scan.cu", "based_norm.cu", "based_embed.cu")]
DEPS = SOURCES + [os.path.join(CSRC, "based_kernels.cuh"), os.path.join(CSRC, "sm103_ptx.cuh"),
                  os.path.join(CSRC, "based_plan.h"), os.path.join(CSRC, "ops_common.cuh"),
                  os.path.join(ROOT, "include", "based.h"), os.path.join(ROOT, "include", "based_ops.h")]
BINDING_SOURCE = os.path.join(CSRC, "ops_binding.cpp")
BINDING_DEPS = [BINDING_SOURCE, os.path.join(ROOT, "include", "based.h"), os.path.join(ROOT, "include", "based_ops.h")]
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC", "-shared", "-Xcompiler", "-fvisibility=hidden",
              "--threads", "0"]  # the sources compile side by side


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _fresh(path: str, deps) -> bool:
    """Whether path exists and is not older than any of deps."""
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def binding_path() -> str:
    """The operators' binding, named by the Python and torch whose interfaces it was compiled against:
    one built for others is not loaded, and is built again."""
    import torch

    tag = "".join(c if c.isalnum() or c in ".+" else "_" for c in torch.__version__)
    return os.path.join(LIB_DIR, f"based_ops_binding-torch{tag}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _binding_commands(obj: str, out: str):
    """The compilation of the binding, and its link against the built library."""
    import torch

    top = os.path.dirname(torch.__file__)
    include = [os.path.join(top, "include"), os.path.join(top, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"), sysconfig.get_paths()["include"]]
    compile_ = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in include:
        compile_ += ["-isystem", d]
    link = ["g++", "-shared", obj, "-o", out, "-L" + LIB_DIR, "-lbased_gb300", "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(top, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return compile_ + ["-c", BINDING_SOURCE, "-o", obj], link


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile the shared library where it is missing or older than any of its sources."""
    os.makedirs(LIB_DIR, exist_ok=True)
    if force or not _fresh(LIB_PATH, DEPS):
        tmp = LIB_PATH + ".tmp"
        cmd = [nvcc()] + NVCC_FLAGS + SOURCES + ["-o", tmp]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB_PATH)
    return LIB_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    """build_library(), and the operators' binding to the library where it is missing or old. The
    library is there even where the binding's compiler, Python's headers or torch are not."""
    os.makedirs(LIB_DIR, exist_ok=True)
    compiler = None
    try:
        path = binding_path()
        obj = path[:-3] + ".o"
        compile_, link = _binding_commands(obj, path + ".tmp")
        if force or not _fresh(path, BINDING_DEPS):
            if verbose:
                print(" ".join(compile_))
            compiler = subprocess.Popen(compile_)  # beside nvcc
    finally:
        try:
            build_library(force, verbose)
        finally:
            failed = compiler is not None and compiler.wait() != 0
    if failed:
        raise subprocess.CalledProcessError(compiler.returncode, compile_)
    if compiler is not None:
        if verbose:
            print(" ".join(link))
        subprocess.run(link, check=True)
        os.replace(path + ".tmp", path)
        os.remove(obj)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
