"""max_ctas caps both of the weighing decode's launches, on the GPU: the grids as a captured graph holds
them."""
import ctypes

import pytest
import torch

import test_gpu_weigh as weigh

pytestmark = pytest.mark.gpu


class KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("smem", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _grids(run):
    """CTAs of each kernel that `run` launches."""
    cu = ctypes.CDLL("libcuda.so.1")
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        run()
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    grids = []
    for node in nodes:
        kind, k = ctypes.c_int(-1), KernelNode()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value == 0:
            assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(k)) == 0
            grids.append(k.grid[0] * k.grid[1] * k.grid[2])
    return grids


@pytest.mark.parametrize("fmt", [None, "e4m3"])
@pytest.mark.parametrize("max_ctas", [1, 7, 100, 300])
def test_max_ctas_caps_both_launches(max_ctas, fmt):
    s = weigh.Step(weigh._hsa(), [900, 64, 3000], 2, 16, 2, fmt)
    out = s.run()
    grids = _grids(lambda: s.run(out=out, max_ctas=max_ctas))
    assert len(grids) == 2 and max(grids) <= max_ctas
    assert len(_grids(lambda: s.run(out=out))) == 2
    s.w.fill_(-7.0)
    s.check(s.run(max_ctas=max_ctas))
