"""Which kernels a call enqueues, by a capture that is never run: for tests of
forms that a rule on sizes chooses."""
from __future__ import annotations

import ctypes
import re

import torch


class _Dim3(ctypes.Structure):
    _fields_ = [("x", ctypes.c_uint32), ("y", ctypes.c_uint32), ("z", ctypes.c_uint32)]


class _KernelNodeParams(ctypes.Structure):
    """hipKernelNodeParams."""
    _fields_ = [("block", _Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", _Dim3), ("params", ctypes.c_void_p),
                ("shared", ctypes.c_uint32)]


def _hip() -> ctypes.CDLL:
    """The HIP runtime that this process has loaded."""
    with open("/proc/self/maps") as f:
        path = next(line.split()[-1] for line in f if "libamdhip64" in line)
    lib = ctypes.CDLL(path)
    lib.hipKernelNameRefByPtr.restype = ctypes.c_char_p
    return lib


def launches(call):
    """[(kernel and its template arguments, workgroups, threads of one)] in
    order, of a call that gets all its tensors from outside."""
    hip = _hip()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t()
    assert hip.hipGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert hip.hipGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    out = []
    for node in nodes:
        p = _KernelNodeParams()
        assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        mangled = hip.hipKernelNameRefByPtr(ctypes.c_void_p(p.func), None).decode()
        name = re.search(r"\d([a-z_]+_kernel)(?:I((?:Li\d+E)+)E)?", mangled)
        args = re.findall(r"\d+", name.group(2) or "")
        out.append((name.group(1) + (f"<{', '.join(args)}>" if args else ""), p.grid.x, p.block.x))
    return out
