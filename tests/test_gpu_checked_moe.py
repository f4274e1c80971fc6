"""The checked build (libdg_debug.so) of routing, the experts' rows, dispatch,
combine and the cross entropy: every form clean under its checks."""
import os
import subprocess
import sys

import pytest

from moe_grouped_gemm_bf16_gb300 import _build

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CASES = '''
import torch
import moe_grouped_gemm_bf16_gb300 as dg
from tests import test_gpu_route as T, test_gpu_expert_rows as E, test_gpu_loss as L

torch.cuda.init()
for sms in (0, 3):
    dg.set_num_sms(sms)
    for case in T.CASES:
        for sigmoid in (False, True):
            T.test_choice_and_weights(case, sigmoid, sigmoid, True, True)
    T.test_values_nearer_than_a_rounding()
    for shape in ((33, 256, 8), (5, 33, 1), (3, 1024, 32)):
        for renorm in (False, True):
            T.test_gradient(shape, False, renorm, renorm)
    for layout in ("ragged", "contiguous", "masked"):
        E.test_rows((2049, 60, 6), layout, True)
        E.test_no_tokens_and_no_choices(layout)
    E.test_dispatch_bf16(65, 2056, 3, 32)
    for ue8m0 in (False, True):
        E.test_dispatch_fp8(33, 640, 3, 8, "masked", ue8m0)
        E.test_dispatch_fp8(300, 1152, 5, 4, "contiguous", ue8m0)
    for shape in E.SUMS:
        E.test_combine(*shape, True, True)
        E.test_combine_gradient(*shape, True)
    for shape in L.SHAPES:
        L.test_loss_and_gradients(shape)
    assert dg.get_device_status() == 0
    dg.set_num_sms(0)
L.test_pieces_of_the_vocabulary((12300, 20001, 64))
for plan in ((True, 256, 256, 2), (False, 192, 64, 4), (False, 256, 128, 1)):
    L.test_every_tiling(plan, (200, 3001, 264))
assert dg.get_device_status() == 0
assert dg.lib()._name.endswith("libdg_debug.so")
print("checked ok")
'''


def test_every_form_runs_clean():
    _build.build(debug=True)
    out = subprocess.run([sys.executable, "-c", CASES], cwd=ROOT, env=dict(os.environ, DG_DEBUG="1"),
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and "checked ok" in out.stdout, out.stdout[-2000:] + out.stderr[-3000:]
