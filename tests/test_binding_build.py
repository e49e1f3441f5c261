"""The compiled binding of the KV cache calls belongs to one torch and one interpreter: it is built again for others, and where it
is missing or foreign the library loads without it (no GPU needed)."""
import os
import shutil
import subprocess
import sys

import pytest

from bit_weight_quantized_matmul_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def test_a_build_for_another_torch_is_not_up_to_date(tmp_path, monkeypatch):
    assert B.up_to_date()
    rebuilt, stamp = [], tmp_path / "for"

    def no_nvcc():
        raise AssertionError("the kernels are up to date")

    monkeypatch.setattr(B, "CALLS_FOR", str(stamp))
    monkeypatch.setattr(B, "build_calls", lambda: rebuilt.append(1))
    monkeypatch.setattr(B, "nvcc", no_nvcc)
    for held in (None, "torch 1.0, CXX11 ABI 0, cpython-38", ""):
        if held is not None:
            stamp.write_text(held)
        assert B.lib_up_to_date() and not B.up_to_date()
        B.build()
    assert len(rebuilt) == 3
    stamp.write_text(B.calls_for())
    B.build()
    assert B.up_to_date() and len(rebuilt) == 3


def test_the_kernels_are_not_built_again_for_the_binding(tmp_path, monkeypatch):
    rebuilt = []
    monkeypatch.setattr(B, "CALLS", str(tmp_path / "_wq_calls.so"))
    monkeypatch.setattr(B, "build_calls", lambda: rebuilt.append(1))
    B.build()
    assert rebuilt == [1]


def in_a_copy(tmp_path, code, calls):
    """Runs `code` beside a copy of the package, with or without its binding."""
    to = tmp_path / "bit_weight_quantized_matmul_gb300"
    to.mkdir()
    for name in ("__init__.py", "build.py", "wq.py", "workloads.py", "libwq.so") + (("_wq_calls.so",) if calls else ()):
        shutil.copy(os.path.join(B.PKG, name), to / name)
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env=dict(os.environ, PYTHONPATH=str(tmp_path)), capture_output=True,
                          text=True, timeout=300)


USE = """
assert wq.lib.wq_packed_bytes(wq.WQ_NF4, 64, 64) == 2048
try:
    wq._calls.attend
except ImportError as e:
    print(e)
"""


def test_without_the_binding_the_linears_work_and_cache_calls_name_the_build(tmp_path):
    r = in_a_copy(tmp_path, "from bit_weight_quantized_matmul_gb300 import wq" + USE, False)
    assert r.returncode == 0, r.stderr
    assert "missing or does not load" in r.stdout and "-m bit_weight_quantized_matmul_gb300.build" in r.stdout


def test_a_binding_for_another_torch_is_not_used(tmp_path):
    r = in_a_copy(tmp_path, "from bit_weight_quantized_matmul_gb300 import build\nbuild.calls_for = lambda: 'torch 9'\n"
                  "from bit_weight_quantized_matmul_gb300 import wq" + USE, True)
    assert r.returncode == 0, r.stderr
    assert f"was built for {B.calls_for()}, this is torch 9" in r.stdout


def test_the_binding_is_for_this_torch():
    from bit_weight_quantized_matmul_gb300 import _wq_calls, wq
    assert wq._calls is _wq_calls and _wq_calls.built_for == B.calls_for()
