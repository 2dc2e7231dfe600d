"""Adapters' gradients where every sum is exact: B_a x and dH keep all 24 bits of binary32 on their
way to dA and dB."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def tokens(g, M, cols):
    """Rows of zeros but for 2^4, 2^-4 and 2^-12 at three columns of their own, and which those are."""
    at = torch.rand(M, cols, generator=g).argsort(1)[:, :3]
    t = torch.zeros(M, cols, dtype=torch.float64)
    t.scatter_(1, at, torch.tensor([2.0 ** 4, 2.0 ** -4, 2.0 ** -12], dtype=torch.float64).expand(M, 3))
    return t, at


def factor(g, L, r, cols, at):
    """Whole numbers below 256 [L, r, cols]; at a row's three columns of its own adapter the first is
    128 or more and the last odd, so that their sum has 24 significant bits, from 2^11 to 2^-12."""
    w = torch.randint(0, 256, (L, r, cols), generator=g).double()
    for a in range(L):
        w[a, :, at[a, 0]] = 128 + w[a, :, at[a, 0]] // 2
        w[a, :, at[a, 2]] = 1 + 2 * (w[a, :, at[a, 2]] // 2)
    sign = torch.randint(0, 2, (L, r, 1), generator=g) * 2 - 1
    return w * sign


@pytest.mark.parametrize("x", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [1, 40, 64, 65, 300, 700])  # few rows up to 64; parts up to 511 / blocks adapters
@pytest.mark.parametrize("d,n,r", [(72, 136, 5), (136, 72, 16), (2056, 2048, 3), (264, 136, 33), (72, 264, 100)])
def test_24_bits(x, M, d, n, r):
    """One row for each adapter: dA = s dY h^T and dB = dh x^T have one term, a power of two times a
    number of 24 bits.  Bit for bit."""
    from integer_rank_adaptation_amd import ops

    g = torch.Generator().manual_seed(M * 7 + r)
    X, at = tokens(g, M, n)
    dY, dat = tokens(g, M, d)
    ids = torch.randperm(M, generator=g)  # row t's adapter; the factors below are by adapter
    of = ids.argsort()
    B = factor(g, M, r, n, at[of])
    A = factor(g, M, r, d, dat[of]).transpose(1, 2).contiguous()
    s = torch.tensor([1.0, -0.5, 4.0])[torch.randint(0, 3, (M,), generator=g)]
    h = (X[of][:, None, :] * B).sum(2)              # [L, r]
    dh = s[:, None].double() * (dY[of][:, :, None] * A).sum(1)
    for v in (h, dh):
        f = v.float()
        assert torch.equal(f.double(), v) and (f.view(torch.int32) & 1).float().mean() > 0.9  # the 24th bit counts
    dA = s[:, None, None].double() * dY[of][:, :, None] * h[:, None, :]
    dB = dh[:, :, None] * X[of][:, None, :]
    dev = [t.to(DT[x]).cuda() for t in (dY, X, A, B)]
    assert all(torch.equal(a.double().cpu(), b) for a, b in zip(dev, (dY, X, A, B)))
    dx, gA, gB = ops.adapters_linear_grad(dev[0], dev[1], ids.int().cuda(), dev[2], dev[3], s.cuda(),
                                          dtype=torch.float32)
    assert torch.equal(gA.cpu().double(), dA) and torch.equal(gB.cpu().double(), dB)
