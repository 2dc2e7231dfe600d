"""The tiled product kernels with contractions of many stages and scale blocks, in every tile
size, against binary64 products (on the GPU, all outputs), under the bounds that
test_gpu_fplinear derives: (K + 16) 2^-23 of the summed magnitudes for the binary32 sums, for
8 bits 7 x 2^-13 of each eight products' largest besides, and one rounding of the output.

Which tiles a size takes (256 compute units) is said at each size.  A contraction of 1104 is nine
stages and scale blocks of 128, the last of 80 columns."""
import numpy as np
import pytest
import torch

from oracle import fplinear as ref
from tests.test_gpu_fplinear import codes_of, offsets_of, ops, randn, rng  # noqa: F401

pytestmark = pytest.mark.gpu

LARGE_AND_QUARTER = (4300, 4096)  # 256 x 256, the last 16 of them cut up, four stages in flight
LARGE_AND_HALF = (5000, 4608)     # 256 x 256, the last 104 of them cut up, two stages in flight
TWO_SETS = (2048, 2048)           # 128 x 128, two sets of waves
ONE_SET = (2100, 2304)            # 128 x 128, two blocks to a unit
SMALL_FOUR_SETS = (1000, 1000)    # 64 x 64, four sets
SMALL_TWO_SETS = (777, 1283)      # 64 x 64, two sets
EVERY_TILE = [LARGE_AND_QUARTER, LARGE_AND_HALF, TWO_SETS, ONE_SET, SMALL_FOUR_SETS, SMALL_TWO_SETS]


def dev64(a):
    return torch.from_numpy(np.asarray(a)).cuda().double()


def values(q, s, rows):
    """The exact values of codes and scale bytes, binary64 on the GPU."""
    return dev64(ref.dequantize(codes_of(q), s.cpu().numpy(), rows))


def aligned(x, w):
    """7 x 2^-13 of the largest product of each group of eight, summed (GPU; the products of two
    codes are exact in binary32)."""
    pad = -x.shape[1] % 8
    x, w = (torch.nn.functional.pad(a.abs(), (0, pad)).float() for a in (x, w))
    total = torch.zeros(x.shape[0], w.shape[0], device="cuda", dtype=torch.float64)
    for j in range(0, x.shape[1], 8):
        m = torch.outer(x[:, j], w[:, j])
        for k in range(j + 1, j + 8):
            torch.maximum(m, torch.outer(x[:, k], w[:, k]), out=m)
        total += m
    return 7 * 2.0**-13 * total


def check(got, x, w, k, what="", eight=False):
    """got against x w^T (binary64) of k terms."""
    if got.numel() == 0:
        return
    want, mag = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
    acc = (k + 16) * 2.0**-23 * mag
    if eight:
        acc += aligned(x, w)
    t = torch.finfo(got.dtype)
    tiny = t.smallest_normal * t.eps / 2 if got.dtype != torch.bfloat16 else 0.0
    bad = ~((got.double() - want).abs() <= acc + t.eps / 2 * (want.abs() + acc) + tiny)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist())


def spread(seed, rows, n, per):
    """Values whose magnitude changes by block of `per` x 128 over 24 binades, so that every
    block dominates some outputs and a scale taken from another one shows."""
    e = rng(seed).integers(-12, 13, (-(-rows // per), -(-n // 128))).astype(np.float32)
    f = torch.from_numpy(np.exp2(e)).repeat_interleave(per, 0)[:rows].repeat_interleave(128, 1)[:, :n]
    return randn(seed + 1, (rows, n)) * f


# --------------------------------------------------------------------------- 8 bits
@pytest.mark.parametrize("M,d", EVERY_TILE)
@pytest.mark.parametrize("n", [1104, 2064])
def test_fp8_every_tile(ops, M, d, n):  # noqa: F811
    xq, sx = ops.fp8_quant_act(spread(M, M, n, 1).cuda())
    w = ops.fp8_quant_weight(spread(d, d, n, 128).cuda())
    Y = ops.fp8_linear(xq, sx, w["wq"], w["sw"])
    check(Y, values(xq, sx, 1), values(w["wq"], w["sw"], 128), n, eight=True)


def _check_groups(Y, off, x, w, n, eight):
    for e in range(len(off) - 1):
        check(Y[off[e]:off[e + 1]], x[off[e]:off[e + 1]], w[e], n, f"group {e}", eight)


# large tiles and their cuts, 4 groups and 70; few rows (the few-row kernel) beside more; two sets
GROUPED = [([1200, 0, 3100, 96], 4096), ([300, 0, 5, 620, 310, 290, 550, 0, 400, 305] * 7, 512),
           ([40, 0, 13, 3] * 20, 300), ([900, 700], 1100)]


@pytest.mark.parametrize("rows,d", GROUPED, ids=lambda v: f"{len(v)}groups" if isinstance(v, list) else str(v))
def test_fp8_grouped_tiles(ops, rows, d):  # noqa: F811
    n, E, lead, tail = 1104, len(rows), 3, 130
    M = lead + sum(rows) + tail
    off = offsets_of(rows, lead)
    xq, sx = ops.fp8_quant_act(spread(M, M, n, 1).cuda())
    w = ops.fp8_quant_weight(torch.stack([spread(e, d, n, 128) for e in range(E)]).cuda())
    out = torch.full((M, d), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = ops.fp8_grouped_linear(xq, sx, off.cuda(), w["wq"], w["sw"], out=out)
    x = values(xq, sx, 1)
    wd = [values(w["wq"][e], w["sw"][e], 128) for e in range(E)]
    _check_groups(Y, off.tolist(), x, wd, n, True)
    assert (Y[:lead] == 7).all() and (Y[M - tail:] == 7).all()


@pytest.mark.parametrize("rows,d,n", [([3, 0, 20, 9], 272, 400), ([300, 0, 150, 33], 1040, 272), ([1500, 900], 1104, 2064)])
def test_fp8_grouped_input_gradient(ops, rows, d, n):  # noqa: F811
    """dX of every group from the transposed codes of its weight [E, n, d]."""
    E, M = len(rows), sum(rows)
    off = offsets_of(rows)
    w = ops.fp8_quant_weight(torch.stack([spread(e + 50, d, n, 128) for e in range(E)]).cuda(), transpose=True)
    dq, sd = ops.fp8_quant_act(spread(M, M, d, 1).cuda())
    dX = ops.fp8_grouped_linear(dq, sd, off.cuda(), w["wq_t"], w["sw_t"])
    wd = [values(w["wq"][e], w["sw"][e], 128).t().contiguous() for e in range(E)]
    _check_groups(dX, off.tolist(), values(dq, sd, 1), wd, d, True)


# --------------------------------------------------------------------------- 16 bits
# rows, d, n: large tiles where there are 4096 columns; of the weight gradient, without a cut
# round and with one; 128 x 128
STEPS = [([2100, 0, 2300, 41], 4096, 1096), ([700, 300, 900, 280], 2304, 2312), ([700, 300, 900, 280], 2296, 2040),
         ([1500, 900], 1544, 1096)]


@pytest.mark.parametrize("rows,d,n", STEPS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_grouped_step_on_large_tiles(ops, dtype, rows, d, n):  # noqa: F811
    """Both types in all directions, the weight gradient in its inputs' type too."""
    M, E = sum(rows), len(rows)
    off = offsets_of(rows)
    X, dY = randn(M, (M, n), 1.0, dtype).cuda(), randn(n, (M, d), 0.1, dtype).cuda()
    W = randn(d, (E, d, n), 0.05, dtype).cuda()
    offd, o = off.cuda(), off.tolist()
    x, dy, w = X.double(), dY.double(), W.double()
    Y, dX = ops.grouped_linear(X, offd, W), ops.grouped_linear_dx(dY, offd, W)
    Wt = W.transpose(1, 2).contiguous()
    Z, dZ = ops.grouped_linear(dY, offd, Wt), ops.grouped_linear_dx(X, offd, Wt)  # the wide side as columns
    dW = [ops.grouped_linear_dw(dY, X, offd, dtype=t) for t in (dtype, torch.float32)]
    dWt = ops.grouped_linear_dw(X, dY, offd)
    for e in range(E):
        r = slice(o[e], o[e + 1])
        we, wt = w[e], w[e].t().contiguous()
        for got, a, b, k, what in ((Y, x, we, n, "Y"), (dX, dy, wt, d, "dX"), (Z, dy, wt, d, "Z"), (dZ, x, we, n, "dZ")):
            check(got[r], a[r], b, k, what)
        dye, xe = dy[r].t().contiguous(), x[r].t().contiguous()
        for got in dW:
            check(got[e], dye, xe, rows[e], "dW")
        check(dWt[e], xe, dye, rows[e], "dW of W^T")
