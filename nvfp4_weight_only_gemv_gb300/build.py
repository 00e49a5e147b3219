"""Builds the CUDA library ``libnvfp4gemv.so`` in-tree for sm_103a with nvcc."""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
SRC = os.path.join(PKG_DIR, "csrc", "nvfp4_gemv.cu")
OPERATORS = tuple(os.path.join(PKG_DIR, "csrc", f) for f in ("rms_norm.cu", "rope_append.cu", "paged_attention.cu"))
HEADER = os.path.join(ROOT, "include", "nvfp4_gemv.h")
BINDING = os.path.join(PKG_DIR, "csrc", "decode_ops_binding.cpp")
SOURCES = (SRC, *OPERATORS, os.path.join(PKG_DIR, "csrc", "ops_common.cuh"), HEADER)
LIB_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(LIB_DIR, "libnvfp4gemv.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the NVFP4 GEMV library needs the CUDA toolkit to build")


def nvcc_command(out: str = LIB_PATH, extra: tuple = (), sources: tuple = (SRC, *OPERATORS), link: bool = True) -> list:
    return [nvcc_path(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xptxas=-warn-spills",
            "-I", os.path.join(ROOT, "include"), "-shared" if link else "-c", "-Xcompiler", "-fPIC",
            *extra, "-o", out, *sources]


def newest_source() -> float:
    return max(os.path.getmtime(f) for f in SOURCES)


def is_stale() -> bool:
    return not os.path.exists(LIB_PATH) or newest_source() > os.path.getmtime(LIB_PATH)


def binding_path() -> str:
    """The binding's file, named after what it is compiled against: this torch and this Python."""
    import torch
    return os.path.join(LIB_DIR, f"_decode_ops.torch-{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def binding_command(out: str) -> list:
    """The Python module that checks the decode operators' tensors, built against the installed torch."""
    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    cuda_inc = [d for d in (os.path.join(cuda, "include"), os.path.join(cuda, "targets", "sbsa-linux", "include"),
                            "/usr/local/cuda/include") if os.path.isdir(d)]
    inc = [os.path.join(ROOT, "include"), os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"], *cuda_inc]
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{d}" for d in inc), "-o", out, BINDING, f"-L{lib}", f"-Wl,-rpath,{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]


def binding_is_stale() -> bool:
    path = binding_path()
    return not os.path.exists(path) or max(map(os.path.getmtime, (BINDING, HEADER))) > os.path.getmtime(path)


def build_binding(force: bool = False) -> str:
    path = binding_path()
    if not force and not binding_is_stale():
        return path
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = path + f".tmp{os.getpid()}"
    cmd = binding_command(tmp)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    os.replace(tmp, path)
    return path


def _compile(out: str, extra: tuple = (), verbose: bool = False) -> None:
    """Compiles each translation unit in a process of its own, all at once, then links them."""
    tag = f".tmp{os.getpid()}"
    objects = [out + "." + os.path.basename(s) + tag + ".o" for s in (SRC, *OPERATORS)]
    cmds = [nvcc_command(o, extra, (s,), link=False) for s, o in zip((SRC, *OPERATORS), objects)]
    try:
        running = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
        said = [p.communicate()[0] for p in running]
        for p, c, text in zip(running, cmds, said):
            if p.returncode != 0:
                raise RuntimeError("nvcc failed:\n" + " ".join(c) + "\n" + text)
        cmd = nvcc_command(out + tag, extra, tuple(objects))
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
        if verbose:
            print("".join(said) + res.stdout + res.stderr)
        os.replace(out + tag, out)
    finally:
        for f in (*objects, out + tag):
            if os.path.exists(f):
                os.remove(f)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if it is missing or older than its sources; return its path."""
    if force or is_stale():
        os.makedirs(LIB_DIR, exist_ok=True)
        _compile(LIB_PATH, verbose=verbose)
    return LIB_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library and the Python binding of the decode operators, where they are missing or
    older than their sources; return the library's path."""
    build_library(force, verbose)
    build_binding(force)
    return LIB_PATH


def variant_path(name: str) -> str:
    return os.path.join(LIB_DIR, f"libnvfp4gemv_{name}.so")


def build_variant(name: str, defines: dict, force: bool = False) -> str:
    """Builds the same source with extra preprocessor definitions (the phase-trace diagnostic,
    planner experiments) into _build/libnvfp4gemv_<name>.so and returns its path. Load it by
    setting NVFP4_GEMV_LIBRARY to that path before the package first loads its library."""
    out = variant_path(name)
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest_source():
        return out
    os.makedirs(LIB_DIR, exist_ok=True)
    _compile(out, tuple(f"-D{k}={v}" for k, v in sorted(defines.items())))
    return out


if __name__ == "__main__":
    print(build(force=True, verbose=True))
