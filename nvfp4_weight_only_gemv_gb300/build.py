"""Builds the CUDA library ``libnvfp4gemv.so`` in-tree for sm_103a with nvcc."""
from __future__ import annotations

import os
import shutil
import subprocess

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
SRC = os.path.join(PKG_DIR, "csrc", "nvfp4_gemv.cu")
OPERATORS = tuple(os.path.join(PKG_DIR, "csrc", f) for f in ("rms_norm.cu", "rope_append.cu", "paged_attention.cu"))
HEADER = os.path.join(ROOT, "include", "nvfp4_gemv.h")
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


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if it is missing or older than its sources; return its path."""
    if not force and not is_stale():
        return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    _compile(LIB_PATH, verbose=verbose)
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
