"""What a call launches: its kernels' grids, blocks and shared memory, read from
a captured graph (nothing runs)."""
import ctypes

import torch


class _Node(ctypes.Structure):
    # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = [("func", ctypes.c_void_p)] + [
        (n, ctypes.c_uint) for n in ("gx", "gy", "gz", "bx", "by", "bz", "smem")] + [
        (n, ctypes.c_void_p) for n in ("params", "extra", "kern", "ctx")]


def launched(call):
    """[(blocks, threads of a block, dynamic shared memory)] of the kernels that
    `call(stream)` launches on the stream it is given.  (Everything that is set
    up on first use has to be: make the call, or a like one, once before.)"""
    cu = ctypes.CDLL("libcuda.so.1")

    def check(r, what):
        assert r == 0, f"{what}: CUresult {r}"

    stream = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    check(cu.cuStreamBeginCapture_v2(handle, 2), "begin capture")
    try:
        call(stream)
    finally:
        check(cu.cuStreamEndCapture(handle, ctypes.byref(graph)), "end capture")
    count = ctypes.c_size_t(0)
    check(cu.cuGraphGetNodes(graph, None, ctypes.byref(count)), "count nodes")
    nodes = (ctypes.c_void_p * count.value)()
    check(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(count)), "get nodes")
    out = []
    for n in nodes:
        p = _Node()
        check(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(n), ctypes.byref(p)), "node")
        out.append((p.gx * p.gy * p.gz, p.bx * p.by * p.bz, p.smem))
    check(cu.cuGraphDestroy(graph), "destroy")
    return out
