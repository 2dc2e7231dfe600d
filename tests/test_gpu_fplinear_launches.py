"""Launches of a call on the floating-point layers, counted in a captured graph."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


def _hip():
    """The HIP runtime that torch has loaded."""
    torch.cuda.init()
    with open("/proc/self/maps") as f:
        path = next(line.split()[-1] for line in f if "libamdhip64" in line)
    return ctypes.CDLL(path)


def launches(call):
    """Kernel nodes of one call."""
    call()  # (first calls set the kernels' attributes)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    n = ctypes.c_size_t(0)
    assert _hip().hipGraphGetNodes(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n)) == 0
    return n.value


def _dense(M, d, n=512):
    from integer_rank_adaptation_amd import ops

    xq, sx = ops.fp8_quant_act(torch.ones(M, n, device="cuda", dtype=torch.bfloat16))
    w = ops.fp8_quant_weight(torch.ones(d, n, device="cuda", dtype=torch.bfloat16))
    out = torch.empty(M, d, device="cuda", dtype=torch.bfloat16)
    return launches(lambda: ops.fp8_linear(xq, sx, w["wq"], w["sw"], out=out)), out


@pytest.mark.parametrize("M,d", [(1, 1024), (128, 512), (129, 511), (129, 1024), (256, 512), (256, 1024), (512, 256),
                                 (1024, 1024)])
def test_a_dense_product_of_one_kind_of_tile_is_one_launch(M, d):
    """Without offsets the row count is known: either the few-row kernel or the tiled one."""
    n, out = _dense(M, d)
    assert n == 1
    assert (out == 512).all()
