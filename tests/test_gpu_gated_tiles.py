"""Gated products on every tile size with contractions of many stages, so that each ring of LDS
buffers is filled again and again within a tile.  Reference in binary64 on the device."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def gate(g, act):
    """(act(g) / g, bound of its relative error): both functions rest on one e^-w, whose argument has
    roundings of w 2^-22, the polynomial and the reciprocal 2^-20; nothing below 2^-126."""
    if act == "silu":
        p, w = torch.sigmoid(g), g.abs()
    else:
        p, w = 0.5 * torch.erfc(-g / math.sqrt(2.0)), 0.5 * g * g
    return p, w * 2.0 ** -22 + 2.0 ** -20 + 2.0 ** -126 / p.clamp(min=1e-200)


def check(got, want, spread, what):
    """Half a step of the type around what lies at most `spread` from `want`."""
    f = torch.finfo(got.dtype)
    tol = spread + f.eps / 2 * (want.abs() + spread).clamp(min=f.tiny)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


# the launches: 64 x 64 tiles with four and two sets of waves, 128 x 128 with two sets and with two blocks
# to a unit, large ones alone (135 to 256), and with a rest of either kind behind them
@pytest.mark.parametrize("T,f", [(400, 320), (1000, 512), (1000, 1160), (2000, 1200), (2300, 1912), (4096, 2048),
                                 (4400, 2048), (5400, 2072)])
@pytest.mark.parametrize("n", [648, 1096])
@pytest.mark.parametrize("x,act,save,groups", [("bf16", "silu", True, 0), ("fp16", "gelu", False, 0),
                                               ("bf16", "gelu", False, 3), ("fp16", "silu", True, 5)])
def test_long_contractions(T, f, n, x, act, save, groups):
    from integer_rank_adaptation_amd import ops

    g = torch.Generator(device="cuda").manual_seed(T + n)
    X = torch.randn(T, n, generator=g, device="cuda").to(DT[x])
    W = (torch.randn(max(groups, 1), 2 * f, n, generator=g, device="cuda") * (2 * n ** -0.5)).to(DT[x])
    cuts = [T * e * e // max(groups, 1) ** 2 for e in range(max(groups, 1) + 1)]  # groups of 1, 3, 5, .. shares
    off = torch.tensor(cuts, device="cuda") if groups else None
    got = ops.gated_linear(X, off, W, act=act, save=save)
    H, GU = got if save else (got, None)
    for e, (a, b) in enumerate(zip(cuts[:-1], cuts[1:])):
        xd, wd = X[a:b].double(), W[e].double().T.contiguous()
        gu = xd @ wd
        # binary32 sums of n products, each step off by 2^-23 of the magnitudes at most
        err = n * 2.0 ** -23 * (xd.abs() @ wd.abs())
        if save:
            check(GU[a:b], gu, err, "projections")
        (gt, up), (eg, eu) = gu.chunk(2, 1), err.chunk(2, 1)
        p, rel = gate(gt, act)
        h = gt * p * up
        check(H[a:b], h, (rel + 2.0 ** -22) * h.abs() + 1.13 * eg * (up.abs() + eu) + (gt * p).abs() * eu, "h")
