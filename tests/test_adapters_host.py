"""Host side of the adapters of many requests (CPU): refusals of the C entry points (nothing
reaches a device), argument checks of the tensor calls, and the plain definition's gradients
against differences."""
import numpy as np
import pytest
import torch

from integer_rank_adaptation_amd import binding as B
from integer_rank_adaptation_amd import ops
from oracle import adapters as ref

P = [0x1000000 * (i + 1) for i in range(16)]  # 16-byte aligned, apart, never dereferenced
OK, EINVAL, ESHAPE, EALIGN, EWS = (B.INTLORA_OK, B.INTLORA_EINVAL, B.INTLORA_ESHAPE, B.INTLORA_EALIGN,
                                   B.INTLORA_EWORKSPACE)


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def _fwd(lib, **kw):
    a = dict(M=8, L=2, d=16, n=1024, r=128, dtype=0, base=P[0], X=P[1], index=P[2], A=P[3], B=P[4], scale=P[5], Y=P[6],
             ws=P[7], size=1 << 22)
    a.update(kw)
    return lib.intlora_adapters_fwd(*a.values(), None)


def _grad(lib, **kw):
    a = dict(M=8, L=2, d=16, n=1024, r=128, dtype=0, out=2, dY=P[8], X=P[1], index=P[2], A=P[3], B=P[4], scale=P[5],
             base=P[0], dX=P[6], dA=P[9], dB=P[10], ws=P[7], size=1 << 22)
    a.update(kw)
    return lib.intlora_adapters_grad(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), EINVAL), (dict(dtype=-1), EINVAL), (dict(r=0), EINVAL), (dict(r=129), EINVAL),
    (dict(L=0), ESHAPE), (dict(L=4097), ESHAPE), (dict(d=12), ESHAPE), (dict(n=20), ESHAPE), (dict(d=0), ESHAPE),
    (dict(n=0), ESHAPE), (dict(M=-1), ESHAPE), (dict(M=1 << 31), ESHAPE), (dict(n=(1 << 20) + 8), ESHAPE),
    (dict(M=(1 << 31) - 300, d=1 << 20), ESHAPE),
    (dict(X=None), EINVAL), (dict(index=None), EINVAL), (dict(A=None), EINVAL), (dict(B=None), EINVAL),
    (dict(scale=None), EINVAL), (dict(ws=None), EWS), (dict(size=64), EWS), (dict(X=P[1] + 8), EALIGN),
    (dict(index=P[2] + 4), EALIGN), (dict(A=P[3] + 2), EALIGN), (dict(base=P[0] + 8), EALIGN),
])
def test_refusals(lib, kw, expect):
    assert _fwd(lib, **kw) == expect
    assert _grad(lib, **kw) == expect
    assert lib.intlora_last_error()


def test_refusals_of_one(lib):
    assert _fwd(lib, Y=None) == EINVAL and _fwd(lib, Y=P[6] + 4) == EALIGN
    assert _fwd(lib, M=0, X=None, Y=None, ws=None) == OK
    assert _grad(lib, dY=None) == EINVAL and _grad(lib, dA=None) == EINVAL and _grad(lib, dB=None) == EINVAL
    assert _grad(lib, dX=None) == EINVAL                 # a base without the dX it belongs to
    assert _grad(lib, out=1) == EINVAL                   # bf16 in, fp16 out
    assert _grad(lib, dA=P[9] + 8) == EALIGN and _grad(lib, dX=P[6] + 2) == EALIGN


@pytest.mark.parametrize("kw", [dict(Y=P[1]), dict(Y=P[0] + 16), dict(Y=P[2]), dict(Y=P[3] + 128), dict(Y=P[4]),
                                dict(Y=P[5]), dict(Y=P[7]), dict(ws=P[1]), dict(ws=P[4] - 256)])
def test_overlaps(lib, kw):
    assert _fwd(lib, **kw) == EINVAL


@pytest.mark.parametrize("kw", [dict(dX=P[1]), dict(dX=P[0] + 16), dict(dA=P[8]), dict(dB=P[9] + 16), dict(dA=P[7]),
                                dict(dB=P[4]), dict(dA=P[3]), dict(ws=P[6])])
def test_overlaps_of_gradients(lib, kw):
    assert _grad(lib, **kw) == EINVAL


def test_workspace(lib):
    f = lib.intlora_adapters_ws_bytes
    assert f(0, 1, 8, 8, 1, 0) == 0
    assert f(1, 0, 8, 8, 1, 0) == 0 and f(1, 1, 8, 12, 1, 0) == 0  # refused sizes
    for M in (1, 17, 1024, 1025, 5000):
        for r in (1, 16, 17, 128):
            small, wide = f(M, 3, 64, 2048, r, 0), f(M, 3, 64, 2048, r, 1)
            need = 4 * M * ((r + 15) // 16 * 16)
            assert wide > need and (small >= need or small == 0)  # 0: one launch, without memory in between


def test_tensor_checks(monkeypatch):
    """The tensor calls look at their arguments before anything else; host tensors are refused."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, ids = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    A, Bm, s = torch.zeros(2, 8, 4, dtype=torch.bfloat16), torch.zeros(2, 4, 16, dtype=torch.bfloat16), torch.zeros(2)
    with pytest.raises(ValueError, match="X: expected a tensor on the current device"):
        ops.adapters_linear(None, x, ids, A, Bm, s)
    with pytest.raises(ValueError, match="A: expected 3 dimensions"):
        ops.adapters_linear(None, x, ids, A[0], Bm, s)

    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)  # as if on the device: the next checks
    good = dict(base=None, X=x, index=ids, A=A, B_=Bm, scale=s)
    for name, t, what in [("index", ids.long(), "torch.int32"), ("index", ids[:3], "shape"),
                          ("A", A.half(), "torch.bfloat16"), ("B_", torch.zeros(2, 5, 16, dtype=torch.bfloat16), "shape"),
                          ("B_", torch.zeros(2, 16, 4, dtype=torch.bfloat16).transpose(1, 2), "contiguous"),
                          ("scale", s.double(), "torch.float32"), ("X", x.float(), "torch.bfloat16"),
                          ("base", torch.zeros(4, 16, dtype=torch.bfloat16), "shape"),
                          ("base", torch.zeros(4, 8), "torch.bfloat16")]:
        with pytest.raises(ValueError, match=what):
            ops.adapters_linear(**{**good, name: t})
    dy = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dtype"):
        ops.adapters_linear_grad(dy, x, ids, A, Bm, s, dtype=torch.float16)
    with pytest.raises(ValueError, match="base"):
        ops.adapters_linear_grad(dy, x, ids, A, Bm, s, base=x, need_dx=False)
    with pytest.raises(ValueError, match="dY"):
        ops.adapters_linear_grad(x, x, ids, A, Bm, s)


def test_definition_against_differences():
    g = np.random.default_rng(3)
    M, L, d, n, r = 7, 3, 8, 16, 3
    base, x, A, Bm = g.normal(size=(M, d)), g.normal(size=(M, n)), g.normal(size=(L, d, r)), g.normal(size=(L, r, n))
    s, dy, index = g.normal(size=L), g.normal(size=(M, d)), np.array([2, 0, 2, -1, 5, 0, 2])
    out, _ = ref.backward(None, dy, x, index, A, Bm, s)
    assert not out["dA"][1].any() and not out["dB"][1].any() and not out["dx"][[3, 4]].any()
    for key, v in (("dx", x), ("dA", A), ("dB", Bm)):
        for at in [tuple(g.integers(0, k) for k in v.shape) for _ in range(12)]:
            keep = v[at]
            v[at] = keep + 1e-5
            hi = (ref.forward(base, x, index, A, Bm, s)[0] * dy).sum()
            v[at] = keep - 1e-5
            lo = (ref.forward(base, x, index, A, Bm, s)[0] * dy).sum()
            v[at] = keep
            # the form is at most quadratic in x or one factor: no truncation, rounding 2^-50 / 1e-5
            assert abs((hi - lo) / 2e-5 - out[key][at]) < 1e-7
