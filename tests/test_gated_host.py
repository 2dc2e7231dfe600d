"""Host side of the gated layer and of the calls on saved codes (CPU): refusals of the C entry
points (nothing reaches a device), argument checks of the tensor calls, and the plain definition's
gradient against differences."""
import numpy as np
import pytest
import torch

from integer_rank_adaptation_amd import binding as B
from integer_rank_adaptation_amd import ops
from oracle import gated as ref

P = [0x1000000 * (i + 1) for i in range(10)]  # 16-byte aligned, apart, never dereferenced
OK, EINVAL, ESHAPE, EALIGN, EWS = (B.INTLORA_OK, B.INTLORA_EINVAL, B.INTLORA_ESHAPE, B.INTLORA_EALIGN,
                                   B.INTLORA_EWORKSPACE)


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def call(fn, defaults, **kw):
    a = {**defaults, **kw}
    assert list(a) == list(defaults)
    return fn(*a.values(), None)


FWD = dict(M=8, E=2, f=16, n=24, dtype=0, act=0, X=P[0], offsets=P[1], W=P[2], H=P[3], GU=P[4])
DGU = dict(M=8, f=16, dtype=1, act=1, dH=P[0], GU=P[1], sGU=P[2], dGU=P[3], H=P[4])
DW = dict(M=8, E=2, d=16, n=32, dtype=0, out=2, dY=P[0], xq=P[1], sx=P[2], offsets=P[3], dW=P[4], ws=P[5], size=512)
RES = dict(M=8, n=32, dtype=2, xq=P[0], sx=P[1], X=P[2])


@pytest.mark.parametrize("kw,expect", [
    (dict(act=2), EINVAL), (dict(act=-1), EINVAL), (dict(dtype=2), EINVAL), (dict(f=12), ESHAPE), (dict(f=-8), ESHAPE),
    (dict(f=(1 << 19) + 8), ESHAPE), (dict(n=20), ESHAPE), (dict(n=0), ESHAPE), (dict(E=0), ESHAPE),
    (dict(E=4097), ESHAPE), (dict(M=-1), ESHAPE), (dict(M=1 << 31), ESHAPE), (dict(offsets=None), EINVAL),
    (dict(X=None), EINVAL), (dict(W=None), EINVAL), (dict(H=None), EINVAL), (dict(GU=P[4] + 8), EALIGN),
    (dict(offsets=P[1] + 8), EALIGN), (dict(H=P[0]), EINVAL), (dict(H=P[2] + 64), EINVAL), (dict(GU=P[3] + 16), EINVAL),
    (dict(GU=P[1]), EINVAL), (dict(M=0, X=None, W=None, H=None), OK), (dict(f=0, X=None, W=None, H=None), OK),
])
def test_forward_refusals(lib, kw, expect):
    assert call(lib.intlora_gated_linear_fwd, FWD, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(act=3), EINVAL), (dict(dtype=2), EINVAL), (dict(f=0), ESHAPE), (dict(f=20), ESHAPE), (dict(M=-1), ESHAPE),
    (dict(M=1 << 31), ESHAPE), (dict(M=(1 << 31) - 1, f=1 << 19), ESHAPE), (dict(f=(1 << 19) + 8), ESHAPE),
    (dict(dH=None), EINVAL), (dict(GU=None), EINVAL), (dict(dGU=None), EINVAL), (dict(sGU=P[2] + 4), EALIGN),
    (dict(dGU=P[0]), EINVAL), (dict(dGU=P[1]), EINVAL), (dict(H=P[0]), EINVAL), (dict(H=P[2]), EINVAL),
    (dict(H=P[3] + 256), EINVAL), (dict(M=0, dH=None, GU=None, dGU=None), OK),
])
def test_backward_refusals(lib, kw, expect):
    assert call(lib.intlora_gated_linear_dgu, DGU, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), EINVAL), (dict(out=1), EINVAL), (dict(n=24), ESHAPE), (dict(d=12), ESHAPE), (dict(E=0), ESHAPE),
    (dict(M=-1), ESHAPE), (dict(offsets=None), EINVAL), (dict(dY=None), EINVAL), (dict(xq=None), EINVAL),
    (dict(sx=None), EINVAL), (dict(dW=None), EINVAL), (dict(sx=P[2] + 4), EALIGN), (dict(dW=P[0]), EINVAL),
    (dict(dW=P[1]), EINVAL), (dict(dW=P[3]), EINVAL), (dict(d=0), OK),
])
def test_dw_refusals(lib, kw, expect):
    assert call(lib.intlora_grouped_linear_dw_fp8, DW, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=3), EINVAL), (dict(n=24), ESHAPE), (dict(n=0), ESHAPE), (dict(M=-1), ESHAPE), (dict(M=1 << 31), ESHAPE),
    (dict(n=(1 << 20) + 16), ESHAPE), (dict(M=(1 << 31) - 1, n=1 << 20), ESHAPE), (dict(xq=None), EINVAL),
    (dict(X=P[2] + 8), EALIGN), (dict(X=P[0]), EINVAL), (dict(X=P[1] - 16), EINVAL), (dict(M=0, xq=None, X=None), OK),
])
def test_restore_refusals(lib, kw, expect):
    assert call(lib.intlora_fp8_dequant_act, RES, **kw) == expect


def test_tensor_checks(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, w = torch.zeros(4, 24, dtype=torch.bfloat16), torch.zeros(2, 32, 24, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="current device"):
        ops.gated_linear(x, off, w)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)  # as if on the device: the next checks
    with pytest.raises(ValueError, match="act"):
        ops.gated_linear(x, off, w, act="relu")
    with pytest.raises(ValueError, match="W: expected shape"):
        ops.gated_linear(x, off, torch.zeros(2, 33, 24, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="offsets"):
        ops.gated_linear(x, None, w)
    with pytest.raises(ValueError, match="torch.int64"):
        ops.gated_linear(x, off.int(), w)
    with pytest.raises(ValueError, match="W: expected torch.bfloat16"):
        ops.gated_linear(x, off, w.half())
    dh = torch.zeros(4, 16, dtype=torch.float16)
    with pytest.raises(ValueError, match="GU: expected torch.float16"):
        ops.gated_linear_dgu(dh, torch.zeros(4, 32))
    with pytest.raises(ValueError, match="GU: expected shape"):
        ops.gated_linear_dgu(dh, torch.zeros(4, 16, dtype=torch.float16))
    q, s = torch.zeros(4, 32, dtype=torch.float8_e4m3fn), torch.zeros(4, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="sGU"):
        ops.gated_linear_dgu(dh, (q, s[:, :1].contiguous()))
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        ops.gated_linear_dgu(dh, (q.view(torch.uint8), s))
    with pytest.raises(ValueError, match="sx"):
        ops.grouped_linear_dw(dh, (q, s[:3]), None)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        ops.grouped_linear_dw(dh, (dh, s), None)
    with pytest.raises(ValueError, match="dtype"):
        ops.grouped_linear_dw(dh, (q, s), None, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dtype"):
        ops.fp8_dequant_act(q, s, torch.float64)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_definition_against_differences(act):
    g = np.random.default_rng(1)
    gu, dh = g.normal(size=(6, 16)) * 2, g.normal(size=(6, 8))
    dgu, h, _, _ = ref.backward(dh, gu, act)
    for at in [(int(g.integers(6)), int(g.integers(16))) for _ in range(40)]:
        vals = []
        for step in (1e-5, -1e-5):
            v = gu.copy()
            v[at] += step
            vals.append((ref.backward(dh, v, act)[1] * dh).sum())
        # third derivatives below 1: truncation 1e-10 |dh u|, rounding 2^-50 / 1e-5
        assert abs((vals[0] - vals[1]) / 2e-5 - dgu[at]) < 1e-8


def test_definition_against_torch():
    g = torch.linspace(-12, 12, 999, dtype=torch.float64)
    for act, fn in (("silu", torch.nn.functional.silu), ("gelu", torch.nn.functional.gelu)):
        x = g.clone().requires_grad_()
        fn(x).sum().backward()
        p, slope, _, _ = ref.gate(g.numpy(), act)
        assert np.allclose(p * g.numpy(), fn(g).numpy(), rtol=1e-9, atol=1e-15)
        assert np.allclose(slope, x.grad.numpy(), rtol=1e-9, atol=1e-14)
