"""Loading the library: the FP8 GEMMs need only libdg.so; the CPython module of
the operators around them belongs to one interpreter and is asked for on the
first call of one of them."""
import importlib.machinery
import os
import subprocess
import sys

import pytest

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def child(code):
    out = subprocess.run([sys.executable, "-c", "import moe_grouped_gemm_bf16_gb300 as dg\n" + code], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    return out.stdout


def test_library_without_the_module():
    out = child("dg.BINDING_PATH = '/nowhere/_binding.so'\n"
                "assert dg.get_tma_aligned_size(3, 4) == 4\n"
                "try: dg.gemm_fp8_fp8_bf16_nt(None, None, 0, None, None, None, 8, 16, 128)\n"
                "except dg.DGError as e: print('status', e.status)\n"
                "try: dg.rms_norm_quantize_fp8_1x128(*[None] * 8, 8, 128, 8, 1e-6)\n"
                "except RuntimeError as e: print('missing', '/nowhere/_binding.so' in str(e))\n")
    assert out.split() == ["status", "1", "missing", "True"]


def test_module_is_this_interpreters():
    assert os.path.exists(dg.BINDING_PATH) and dg.BINDING_PATH == _build.BINDING
    assert os.path.basename(dg.BINDING_PATH) == "_binding" + importlib.machinery.EXTENSION_SUFFIXES[0]
    assert "cpython" in dg.BINDING_PATH
    from moe_grouped_gemm_bf16_gb300 import _binding
    assert _binding.__file__ == dg.BINDING_PATH


def test_build_without_python_headers(tmp_path, monkeypatch):
    """The library is built all the same, with a warning that says what is missing."""
    old = tmp_path / "_binding.so"   # of an older header: not to be called
    old.write_bytes(b"")
    os.utime(old, (0, 0))
    monkeypatch.setattr(_build, "BINDING", str(old))
    monkeypatch.setattr(_build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "no headers")})
    monkeypatch.setenv("CPATH", "")
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.listdir(tmp_path)
