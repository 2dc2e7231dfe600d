"""Refusals of the sum of squared gradients whose sum or workspace lies in another of the call's
buffers (CPU: every call below ends in validation, nothing reaches a device), and what is no
overlap."""
import ctypes

import pytest
import torch

from integer_rank_adaptation_amd import binding as B

G0, G1, SUM, WS = 0x100000, 0x200000, 0x300000, 0x400000
NUMEL = (100, 40000)  # fp32 and bf16: 400 and 80000 bytes; 1 + 3 partial sums of 8 bytes


def _sumsq(sumsq, ws, ws_bytes=32):
    p, n, t = (ctypes.c_void_p * 2)(G0, G1), (ctypes.c_int64 * 2)(*NUMEL), (ctypes.c_int32 * 2)(2, 0)
    return B.lib().intlora_grad_sumsq(2, p, n, t, sumsq, ws, ws_bytes, None)


@pytest.mark.parametrize("sumsq,ws", [
    (G0, WS), (G0 + 384, WS), (G1 + 79984, WS),          # the sum in a gradient: first, last bytes
    (SUM, G0), (SUM, G1), (SUM, G0 - 16), (SUM, G1 + 79984),  # partial sums in one, or running into it
    (WS, WS), (WS + 16, WS),                              # the sum among the partial sums
])
def test_sum_and_workspace_lie_apart(sumsq, ws):
    assert _sumsq(sumsq, ws) == B.INTLORA_EINVAL
    assert b"overlaps" in B.lib().intlora_last_error()


def _dw_without_rows(E, d, n, tokens, out):
    """Weight gradients of empty groups: the token operands have no elements."""
    return B.lib().intlora_grouped_linear_dw(0, E, d, n, 0, 0, tokens, tokens, None, out, None)


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the made-up addresses would be written to")
def test_tensors_without_elements_overlap_nothing():
    assert _dw_without_rows(1, 16, 16, G0 + 64, G0) == B.INTLORA_EDEVICE  # past validation, no GPU here


@pytest.mark.gpu
def test_weight_gradient_without_rows_inside_its_output():
    out = torch.full((1, 16, 16), 3.0, dtype=torch.bfloat16, device="cuda")
    assert _dw_without_rows(1, 16, 16, out.data_ptr() + 64, out.data_ptr()) == B.INTLORA_OK
    torch.cuda.synchronize()
    assert not out.any()
