"""The kernels of a call: what it captures into a CUDA graph, node by node, with names and grids."""
from __future__ import annotations

import ctypes
import re

import torch


class _Kernel(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def kernels(call) -> list[tuple[str, tuple[int, int, int], tuple[int, int, int]]]:
    """(mangled name, grid, block) of every kernel that ``call`` launches on the current stream.  It is
    captured, not run; call it once before, so that nothing is set up under the capture."""
    cuda = ctypes.CDLL("libcuda.so.1")

    def do(name, *args):
        assert getattr(cuda, name)(*args) == 0, name
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g):
        call()
    graph = ctypes.c_void_p(g.raw_cuda_graph())
    n = ctypes.c_size_t()
    do("cuGraphGetNodes", graph, None, ctypes.byref(n))
    nodes = (ctypes.c_void_p * n.value)()
    do("cuGraphGetNodes", graph, nodes, ctypes.byref(n))
    out = []
    for node in nodes:
        kind = ctypes.c_int()
        do("cuGraphNodeGetType", ctypes.c_void_p(node), ctypes.byref(kind))
        if kind.value != 0:  # (a kernel's)
            continue
        k, name = _Kernel(), ctypes.c_char_p()
        do("cuGraphKernelNodeGetParams_v2", ctypes.c_void_p(node), ctypes.byref(k))
        if k.kern:
            do("cuKernelGetName", ctypes.byref(name), ctypes.c_void_p(k.kern))
        else:
            do("cuFuncGetName", ctypes.byref(name), ctypes.c_void_p(k.func))
        out.append((name.value.decode(), tuple(k.grid), tuple(k.block)))
    return out


def variants(call, *wanted: str) -> list[tuple[str, tuple[int, ...], tuple[int, int, int]]]:
    """(kernel, template numbers, grid) of the call's launches of the kernels named, in order."""
    out = []
    for name, grid, _ in kernels(call):
        for kernel in wanted:
            m = re.search(rf"{len(kernel)}{kernel}(I(?:L[a-z]n?\d+E)+)?", name)
            if m:
                numbers = re.findall(r"L[a-z](n?)(\d+)E", m.group(1) or "")
                out.append((kernel, tuple(-int(v) if minus else int(v) for minus, v in numbers), grid))
    return out
