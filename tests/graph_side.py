"""Which kernels a call launches: the call is captured, and the graph's nodes are read."""
from __future__ import annotations

import ctypes

import torch

KERNELS = ("decode_fp4_kernel", "prefill_fp4_kernel", "prefill_plan_kernel")


class _Params(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3),
                ("block", ctypes.c_uint * 3), ("smem", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


class Captured:
    """``call`` captured: ``kernels`` lists (name, grid, cluster) of its launches;
    ``replay`` runs it."""

    def __init__(self, call):
        self.graph = torch.cuda.CUDAGraph(keep_graph=True)
        torch.cuda.synchronize()
        with torch.cuda.graph(self.graph):
            call()
        self.kernels = _kernels(self.graph.raw_cuda_graph())
        self.graph.instantiate()
        self.replay = self.graph.replay

    def of(self, name):
        """The launches of one kernel."""
        return [k for k in self.kernels if k[0] == name]


def _kernels(graph):
    cu = ctypes.CDLL("libcuda.so.1")

    def ok(status):
        if status:
            raise RuntimeError(f"driver call failed: {status}")

    graph, n = ctypes.c_void_p(graph), ctypes.c_size_t(0)
    ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
    nodes = (ctypes.c_void_p * n.value)()
    ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
    out = []
    for node in nodes:
        node, kind = ctypes.c_void_p(node), ctypes.c_int(-1)
        ok(cu.cuGraphNodeGetType(node, ctypes.byref(kind)))
        if kind.value != 0:  # not a kernel
            continue
        p = _Params()
        ok(cu.cuGraphKernelNodeGetParams_v2(node, ctypes.byref(p)))
        text = ctypes.c_char_p()
        if p.func:
            ok(cu.cuFuncGetName(ctypes.byref(text), ctypes.c_void_p(p.func)))
        else:
            ok(cu.cuKernelGetName(ctypes.byref(text), ctypes.c_void_p(p.kern)))
        value = (ctypes.c_uint * 16)()  # CUlaunchAttributeValue, 64 bytes
        ok(cu.cuGraphKernelNodeGetAttribute(node, 4, value))  # cluster dimension
        mangled = text.value.decode()
        name = next((k for k in KERNELS if f"{len(k)}{k}" in mangled), mangled)
        out.append((name, int(p.grid[0]), max(int(value[0]), 1)))
    return out
