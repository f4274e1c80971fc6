"""The example's decoding step refuses a batch that could overflow an expert's
rows before anything runs (an index past them would end the process on the GPU)."""
import importlib.util
import os
import types

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_batch_larger_than_an_experts_rows():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    w = types.SimpleNamespace(hidden=256, inter=128, experts=4)
    x = torch.zeros(129, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="129 tokens"):
        layer.decode_step(w, None, None, x, x, top_k=2, max_m=128)
