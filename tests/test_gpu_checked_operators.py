"""The checked build (libdg_debug.so) of the operators around the GEMMs: the
checks by themselves, and every form clean under them."""
import os
import subprocess
import sys

import pytest

from moe_grouped_gemm_bf16_gb300 import _build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_checks(tmp_path):
    exe = str(tmp_path / "helpers")
    r = subprocess.run([_build.nvcc(), "-std=c++17", "-O2", "-DDG_DEBUG=1", *_build.ARCH, "-I", _build.CSRC, "-I",
                        _build.INCLUDE, os.path.join(ROOT, "tests", "checked_helpers.cu"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, (out.returncode, out.stderr)
    # result, then (status, abort flag)
    assert [int(v) for v in out.stdout.split()] == [
        1, 0, 0,    0, 11, 0,    0, 11, 0,    0, 11, 0,   # in_bounds: inside, across, behind, wrapping around
        1, 1, 0, 0,    0, 12, 1,                          # the first fill; not a second one
        1, 11, 1,                                         # past the operand: not loaded
        3, 1, 1, 0, 0,                                    # its last, shorter chunk
        11, 1]                                            # before the operand


CASES = '''
import torch
import moe_grouped_gemm_bf16_gb300 as dg
from tests import test_gpu_norm as N, test_gpu_swiglu as S, test_gpu_bf16_few_rows as F
from tests import test_gpu_bf16_ragged as P, test_gpu_sm_limit as L, test_gpu_swiglu_ring as A

for sms in (0, 3):
    dg.set_num_sms(sms)
    for M, K, ld in ((7, 1536, 8), (700, 384, 700), (1900, 7168, 1900), (40, 16384, 40)):
        for ue8m0 in (False, True):
            X, Rs, W = N.normal(M, K, seed=M), N.normal(M, K, seed=K, scale=3.0), N.normal(K, seed=1)
            N.check(X, Rs, W, N.forward(X, Rs, W, M, K, ld, ue8m0), M, K, ue8m0, "HYQr", "norm")
            assert dg.get_device_status() == 0, (M, K)
    for M, K in ((33, 640), (611, 384), (1000, 4224), (500, 16384)):
        H, W = N.normal(M, K, seed=M, scale=2.0), N.normal(K, seed=K, scale=0.5)
        dY, rstd = N.normal(M, K, seed=M + 1, scale=0.03), torch.rsqrt(H.float().square().mean(-1) + N.EPS)
        first = N.backward(dY, H, rstd, W, None)
        assert all(torch.isfinite(t.float()).all() for t in first) and dg.get_device_status() == 0, (M, K)
    for shape in ((1, 37, 256), (1, 11003, 2048), (3, 700, 4224)):
        for ue8m0 in (False, True):
            a = A.Activation(*shape, ue8m0, "YQC", seed=sum(shape))
            a()
            a.check()
    S.test_swiglu_gradient((3, 64, 384), [64, 0, 33])
    for form in ("nt", "nn", "tn"):
        for sizes, n, k in (([1, 0, 2], 136, 520), ([40, 0, 24], 520, 4104), ([600, 300], 392, 264)):
            x, y = P.inputs(form, sizes, n, k, seed=n)
            P.check(form, x, y, sizes, P.run(form, x, y, sizes, n), form)
    dg.set_num_sms(0)
assert dg.lib()._name.endswith("libdg_debug.so")
print("checked ok")
'''


def test_every_form_runs_clean():
    _build.build(debug=True)
    out = subprocess.run([sys.executable, "-c", CASES], cwd=ROOT, env=dict(os.environ, DG_DEBUG="1"),
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and "checked ok" in out.stdout, out.stdout[-2000:] + out.stderr[-3000:]
