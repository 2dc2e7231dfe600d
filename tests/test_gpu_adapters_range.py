"""Adapters whose ranks differ widely in size: a rank that is small beside the token's largest one
keeps its bits where an output depends on it alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(v, dtype):
    f = torch.finfo(dtype)
    return f.eps / 2 * v.abs().clamp(min=f.tiny)


def spread_factors(g, L, d, n, r, dt):
    """B's row k is 2^-k as large as its first, and each of A's rows has one number, in column
    i % r, 2^k as large: outputs of about unit size that hang on one rank each."""
    k = torch.arange(r)
    B = (torch.randn(L, r, n, generator=g).double() * 2.0 ** (6.0 - k)[None, :, None]).to(dt)
    A = torch.zeros(L, d, r, dtype=dt)
    i = torch.arange(d)
    A[:, i, i % r] = ((torch.rand(L, d, generator=g).double() + 0.5) * 2.0 ** (i % r - 10.0)).to(dt)
    return A, B


def near(got, want, e, what):
    off = ((got.double() - want).abs() / (e + half_step(want.abs() + e, got.dtype))).max().item()
    assert off <= 1, f"{what}: {off:.3g} times the bound"


def terms(t, first, second, s):
    """s_a second (first t) of a token row, and the bound of its error before the last rounding: the
    first sum 2^-23 of its magnitudes for each product, 16 bits of it, four steps after that."""
    h, wide = first @ t, first.abs() @ t.abs()
    y = s * (second @ h)
    e = second.abs() @ (t.numel() * 2.0 ** -23 * wide + 2.0 ** -16 * h.abs())
    return y, abs(s) * e + 4 * 2.0 ** -23 * y.abs()


@pytest.mark.parametrize("x", ["fp16", "bf16"])
@pytest.mark.parametrize("M,L,d,n,r", [
    (5, 2, 264, 72, 16),       # one launch
    (40, 3, 264, 136, 20),     # few rows
    (700, 3, 264, 136, 20),    # listed rows
    (900, 2, 1032, 2056, 21),  # splits of the columns, padded factors
])
def test_small_ranks(x, M, L, d, n, r):
    from integer_rank_adaptation_amd import ops

    dt = DT[x]
    g = torch.Generator().manual_seed(M + r)
    X = torch.randn(M, n, generator=g).to(dt)
    A, B = spread_factors(g, L, d, n, r, dt)
    s = torch.rand(L, generator=g) + 0.5
    ids = torch.randint(0, L, (M,), generator=g, dtype=torch.int32)
    y = ops.adapters_linear(None, X.cuda(), ids.cuda(), A.cuda(), B.cuda(), s.cuda()).cpu()
    for t in range(M):
        a = int(ids[t])
        want, e = terms(X[t].double(), B[a].double(), A[a].double(), float(s[a]))
        near(y[t], want, e, f"row {t} of adapter {a}")


@pytest.mark.parametrize("x", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [40, 700])
def test_small_ranks_of_the_input_gradient(x, M):
    """dX of factors the other way round: B^T's rows hold one number each, dH spans the range."""
    from integer_rank_adaptation_amd import ops

    dt, L, d, n, r = DT[x], 3, 136, 264, 20
    g = torch.Generator().manual_seed(M)
    Bt, At = spread_factors(g, L, n, d, r, dt)  # [L, n, r] and [L, r, d]
    A, B = At.transpose(1, 2).contiguous(), Bt.transpose(1, 2).contiguous()
    dY, X = torch.randn(M, d, generator=g).to(dt), torch.randn(M, n, generator=g).to(dt)
    s = torch.rand(L, generator=g) + 0.5
    ids = torch.randint(0, L, (M,), generator=g, dtype=torch.int32)
    dx = ops.adapters_linear_grad(dY.cuda(), X.cuda(), ids.cuda(), A.cuda(), B.cuda(), s.cuda())[0].cpu()
    for t in range(M):
        a = int(ids[t])
        want, e = terms(dY[t].double(), At[a].double(), Bt[a].double(), float(s[a]))
        near(dx[t], want, e, f"row {t} of adapter {a}")
