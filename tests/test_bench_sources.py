"""The code that a traffic record belongs to: what the workload's kernels include,
however deep, and nothing of the others."""
import os
import shutil

import pytest

from tests.test_bench_helpers import ROOT, _bench

CSRC = os.path.join("moe_grouped_gemm_bf16_gb300", "csrc")


@pytest.fixture
def bench(tmp_path):
    shutil.copytree(os.path.join(ROOT, CSRC), tmp_path / CSRC)
    b = _bench()
    b.ROOT = str(tmp_path)
    return b


def changed(b, name):
    """Workloads whose hash a change of the file's code changes."""
    before = {w: b.kernel_source_hash(w) for w in ("quantize_act", "dense_decode", "grouped_masked")}
    path = os.path.join(b.ROOT, CSRC, name)
    with open(path, "a") as f:
        f.write("\nint changed;\n")
    return {w for w, h in before.items() if b.kernel_source_hash(w) != h}


GEMMS = {"dense_decode", "grouped_masked"}


@pytest.mark.parametrize("name,want", [
    ("dg_quant.cu", {"quantize_act"}), ("dg_quant.h", {"quantize_act"}), ("dg_fp8.cuh", {"quantize_act"}),
    ("dg_kernel.cuh", GEMMS), ("dg_kernel_bs.cuh", GEMMS), ("dg_instances.cuh", GEMMS), ("ptx.cuh", GEMMS),
    ("dg_wait.cuh", GEMMS), ("dg_params.h", GEMMS), ("dg_inst_masked.cu", GEMMS),
    ("dg_host.cu", GEMMS | {"quantize_act"}), ("dg_norm.cu", set()), ("dg_ring.cuh", set()),
    ("dg_launch.h", set()), ("dg_bf16.cu", set()), ("dg_ops_host.cu", set()), ("dg_ops_binding.cpp", set())])
def test_changes_count_where_they_are_compiled_in(bench, name, want):
    assert changed(bench, name) == want


def test_comments_do_not_count(bench):
    h = bench.kernel_source_hash("quantize_act")
    with open(os.path.join(bench.ROOT, CSRC, "dg_fp8.cuh"), "a") as f:
        f.write("\n// a remark\n/* and\n another */\n")
    assert bench.kernel_source_hash("quantize_act") == h
