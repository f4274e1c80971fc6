"""The cross entropy of up to 64 tokens in tiles of every multiple of 32 words: the
tensor cores take 128 lanes at a time, so that the operand of 96, 160 or 224 words is read past
its end (into what lies behind it in shared memory), and what comes of that is dropped."""
import os
import subprocess
import sys

import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests.test_gpu_loss import backward, check_backward, check_forward, forward, inputs

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHAPES = [(40, 3001, 1040), (64, 700, 1024), (3, 20011, 1096), (16, 5000, 72), (1, 159, 2048), (33, 225, 136)]


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()
    yield
    assert dg.get_device_status() == 0


@pytest.mark.parametrize("lanes,rows", [(96, 64), (160, 64), (224, 64), (160, 128), (224, 128)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_tiles_of_multiples_of_32_words(lanes, rows, shape):
    X, W, t, d = inputs(*shape, seed=lanes)
    t[0] = min(shape[1] - 1, lanes - 1)    # (the last word of a tile)
    dg.debug_force_ragged_plan(False, lanes, rows, 1)
    try:
        loss, lse = forward(X, W, t)
        dX, dW = backward(X, W, t, lse, d)
    finally:
        dg.debug_force_ragged_plan()
    check_forward(X, W, t, loss, lse)
    check_backward(X, W, t, lse, d, dX, dW)


def test_more_tokens_take_multiples_of_64_only():
    X, W, t, _ = inputs(65, 300, 64, seed=2)
    dg.debug_force_ragged_plan(False, 160, 64, 1)
    try:
        with pytest.raises(dg.DGError) as e:
            forward(X, W, t)
    finally:
        dg.debug_force_ragged_plan()
    assert e.value.status == 2


def test_the_estimates_own_choice():
    # sizes for which the estimate takes tiles of 160 and of 224 words (as many tiles as make whole
    # waves), without a forced plan
    for T, V, K in ((16, 24300, 2048), (61, 34000, 1024), (9, 48600, 1024), (50, 32000, 2048)):
        X, W, t, d = inputs(T, V, K, seed=V)
        loss, lse = forward(X, W, t)
        check_forward(X, W, t, loss, lse)
        check_backward(X, W, t, lse, d, *backward(X, W, t, lse, d))


CHECKED = '''
import torch
import moe_grouped_gemm_bf16_gb300 as dg
from tests import test_gpu_loss_tiles as L

torch.cuda.init()
for shape in L.SHAPES:
    for plan in ((96, 64), (160, 64), (224, 64), (160, 128), (224, 128)):
        L.test_tiles_of_multiples_of_32_words(*plan, shape)
assert dg.get_device_status() == 0 and dg.lib()._name.endswith("libdg_debug.so")
print("checked ok")
'''


def test_every_tile_runs_clean():
    _build.build(debug=True)
    out = subprocess.run([sys.executable, "-c", CHECKED], cwd=ROOT, env=dict(os.environ, DG_DEBUG="1"),
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and "checked ok" in out.stdout, out.stdout[-2000:] + out.stderr[-3000:]
