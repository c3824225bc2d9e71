"""What a call launches: the call is captured into a graph, which is looked at and thrown away, so
nothing runs.  Tests use it to see that the sizes they compare reach the kernel they mean."""
from __future__ import annotations

import ctypes
import re
from typing import NamedTuple

import torch


class Launch(NamedTuple):
    name: str        # mangled
    grid: tuple
    threads: int
    cluster: int     # blocks of a cluster, 1: none

    @property
    def numbers(self) -> tuple:
        """The kernel's whole-number and truth-valued template arguments, in their order."""
        return tuple(int(v) for v in re.findall(r"L[ib](\d+)E", self.name))


class _Params(ctypes.Structure):   # CUDA_KERNEL_NODE_PARAMS_v2
    _fields_ = ([("func", ctypes.c_void_p)] + [(n, ctypes.c_uint) for n in (
        "gx", "gy", "gz", "bx", "by", "bz", "smem")] + [(n, ctypes.c_void_p) for n in (
            "params", "extra", "kern", "ctx")])


_CLUSTER_DIMENSION = 4   # CU_LAUNCH_ATTRIBUTE_CLUSTER_DIMENSION


def _do(status):
    assert status == 0, f"CUDA driver status {status}"


def captured(call) -> list[Launch]:
    """The kernels that call(stream) enqueues on the stream it is given."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream = torch.cuda.Stream()
    handle = ctypes.c_void_p(stream.cuda_stream)
    graph = ctypes.c_void_p()
    _do(cu.cuStreamBeginCapture_v2(handle, 2))
    try:
        call(stream)
    finally:
        status = cu.cuStreamEndCapture(handle, ctypes.byref(graph))
    _do(status)
    try:
        n = ctypes.c_size_t()
        _do(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
        nodes = (ctypes.c_void_p * n.value)()
        _do(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
        out = []
        for node in nodes:
            p = _Params()
            _do(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(p)))
            name = ctypes.c_char_p()
            if p.func:
                _do(cu.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(p.func)))
            else:
                _do(cu.cuKernelGetName(ctypes.byref(name), ctypes.c_void_p(p.kern)))
            value = (ctypes.c_uint * 16)()
            _do(cu.cuGraphKernelNodeGetAttribute(ctypes.c_void_p(node), _CLUSTER_DIMENSION, value))
            out.append(Launch(name.value.decode(), (p.gx, p.gy, p.gz), p.bx, max(1, value[0])))
        return out
    finally:
        cu.cuGraphDestroy(graph)


def launch_of(call) -> Launch:
    """The one kernel that call(stream) enqueues."""
    found = captured(call)
    assert len(found) == 1, found
    return found[0]
