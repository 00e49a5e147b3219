"""What loads when only a part of the compiled files is there, in a copy of the package without a compiler."""
import os
import shutil
import subprocess
import sys

import pytest

import nvfp4_weight_only_gemv_gb300 as nv
from nvfp4_weight_only_gemv_gb300 import build

NO_COMPILER = """
import nvfp4_weight_only_gemv_gb300.build as b
def missing():
    raise RuntimeError("nvcc not found")
b.nvcc_path = missing
import nvfp4_weight_only_gemv_gb300 as nv, torch
assert nv.__file__.startswith({root!r}), nv.__file__
"""


@pytest.fixture
def copy(tmp_path):
    """run(code): runs code in a copy of the package that has the library, without a compiler."""
    nv.library()
    name = os.path.basename(build.PKG_DIR)
    skip = shutil.ignore_patterns("__pycache__", "_decode_ops*", "*.tmp*")
    shutil.copytree(build.PKG_DIR, tmp_path / name, ignore=skip)
    shutil.copytree(os.path.join(build.ROOT, "include"), tmp_path / "include")

    def run(code):
        env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
        return subprocess.run([sys.executable, "-c", NO_COMPILER.format(root=str(tmp_path)) + code], cwd=tmp_path, env=env,
                              capture_output=True, text=True, timeout=250)

    run.root, run.package = tmp_path, tmp_path / name
    return run


def test_the_products_load_without_the_decode_operators_binding(copy):
    out = copy("nv.library(); print(nv.describe_plan_host('dense', 1, 4096, 4096))")
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.strip()


def test_the_decode_operators_name_what_is_missing(copy):
    out = copy("""
try:
    nv.rms_norm(torch.zeros(1, 8), torch.ones(8))
except RuntimeError as e:
    print(e)
""")
    assert out.returncode == 0 and "nvcc not found" in out.stdout, out.stderr[-2000:]


def test_an_older_library_serves_where_no_compiler_is(copy):
    os.utime(copy.root / "include" / "nvfp4_gemv.h")  # every compiled file is now stale
    out = copy("print(nv.describe_plan_host('dense', 1, 4096, 4096))")
    assert out.returncode == 0, out.stderr[-2000:]


def test_an_older_binding_serves_where_no_compiler_is(copy):
    shutil.copy2(build.build_binding(), copy.package / "_build")
    os.utime(copy.root / "include" / "nvfp4_gemv.h")
    out = copy("""
try:
    nv.rms_norm(torch.zeros(1, 8), torch.ones(8))
except ValueError as e:
    print(e)
""")
    assert out.returncode == 0 and "CUDA tensor" in out.stdout, out.stderr[-2000:]


def test_a_binding_for_another_torch_or_python_does_not_serve(monkeypatch):
    import sysconfig

    import torch
    build.build_binding()
    assert not build.binding_is_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.0.0+other")
        assert build.binding_is_stale()
    with monkeypatch.context() as m:
        known = sysconfig.get_config_var
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-39-other" if name == "SOABI" else known(name))
        assert build.binding_is_stale()
    assert not build.binding_is_stale()


def test_threads_build_the_binding_once(monkeypatch):
    import threading
    import time

    from nvfp4_weight_only_gemv_gb300 import decode_ops
    build.build_binding()
    inside, most, calls = [0], [0], [0]

    def slow(force=False):
        inside[0] += 1
        calls[0] += 1
        most[0] = max(most[0], inside[0])
        time.sleep(0.2)
        inside[0] -= 1
        return build.binding_path()

    monkeypatch.setattr(build, "build_binding", slow)
    monkeypatch.setattr(decode_ops, "_native", decode_ops._Unbound())
    threads = [threading.Thread(target=decode_ops._load) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert most[0] == 1 and calls[0] == 1
