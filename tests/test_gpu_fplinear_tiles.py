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


# --------------------------------------------------------------------------- what lies beside
def _same_elsewhere(dirty, clean, rows):
    keep = torch.ones(clean.shape[0], dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.isfinite(clean).all() and torch.equal(dirty[keep], clean[keep])


@pytest.mark.parametrize("M,d", EVERY_TILE)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_fp8_nonfinite_blocks_in_tiles(ops, M, d, bad):  # noqa: F811
    """A token block that holds a NaN or infinity makes its row NaN and changes no other output;
    a weight block its 128 outputs.  Bad blocks at a row's start follow the row before's tail."""
    n = 208
    X, W = randn(M, (M, n)).cuda(), randn(d, (d, n), 0.02).cuda()
    w = ops.fp8_quant_weight(W)
    Y = ops.fp8_linear(*ops.fp8_quant_act(X), w["wq"], w["sw"])
    rows = torch.tensor([5, 63, 64, 130, 255, 256, M - 300, M - 1], device="cuda")
    Xb = X.clone()
    Xb[rows, torch.tensor([0, 3, 207, 127, 128, 0, 60, 200], device="cuda")] = bad
    xq, sx = ops.fp8_quant_act(Xb)
    assert (sx == 255).sum() == len(rows)
    Yb = ops.fp8_linear(xq, sx, w["wq"], w["sw"])
    assert torch.isnan(Yb[rows]).all()
    _same_elsewhere(Yb, Y, rows)
    Wb = W.clone()
    Wb[300, 5] = Wb[d - 1, 207] = bad
    w = ops.fp8_quant_weight(Wb)
    cols = torch.cat([torch.arange(256, 384), torch.arange((d - 1) // 128 * 128, d)]).cuda()
    Yb = ops.fp8_linear(*ops.fp8_quant_act(X), w["wq"], w["sw"])
    assert torch.isnan(Yb[:, cols]).all()
    _same_elsewhere(Yb.t(), Y.t(), cols)


# tiles of the products: 64 x 64 and 128 x 128 in sets, 128 x 128, large ones and their cuts
BESIDE = [([300, 150, 400], 1096), ([600, 300, 600], 1504), ([500, 200, 500], 4096), ([2100, 196, 2100], 4096)]


@pytest.mark.parametrize("rows,d", BESIDE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_nan_of_one_group_in_tiles(ops, dtype, rows, d):  # noqa: F811
    """NaN tokens and infinite weights of the middle group change no output of the others, although
    tiles reach over the groups' borders and the ends of rows (72 columns: half a stage)."""
    n, M = 72, sum(rows)
    off = offsets_of(rows)
    mid = torch.arange(int(off[1]), int(off[2]), device="cuda")
    X, dY = randn(1, (M, n), 1.0, dtype).cuda(), randn(2, (M, d), 0.1, dtype).cuda()
    W = randn(3, (3, d, n), 0.05, dtype).cuda()
    Wt = W.transpose(1, 2).contiguous()
    offd = off.cuda()

    def run(x, dy, w, wt):
        return [ops.grouped_linear(x, offd, w), ops.grouped_linear_dx(x, offd, wt), ops.grouped_linear(dy, offd, wt),
                ops.grouped_linear_dx(dy, offd, w)], [ops.grouped_linear_dw(dy, x, offd), ops.grouped_linear_dw(x, dy, offd)]

    clean, clean_dw = run(X, dY, W, Wt)
    Xb, dYb, Wb = X.clone(), dY.clone(), W.clone()
    Xb[mid], dYb[mid], Wb[1] = float("nan"), float("inf"), float("inf")
    dirty, dirty_dw = run(Xb, dYb, Wb, Wb.transpose(1, 2).contiguous())
    for a, b in zip(dirty, clean):
        _same_elsewhere(a, b, mid)
        assert not torch.isfinite(a[mid]).any()
    for a, b in zip(dirty_dw, clean_dw):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]) and torch.isnan(a[1]).all()


def _wild_offsets(seed, E, M):
    """Offsets that ascend on the whole, with entries far outside [0, M] and below their predecessors."""
    g = rng(seed)
    off = np.sort(g.integers(0, M + 1, E + 1)).astype(np.int64)
    off[0] = -(1 << 40)
    at = g.permutation(np.arange(1, E))
    k = max(1, E // 6)
    off[at[:k]] -= g.integers(1, M, k)          # descending, some below 0
    off[at[k:2 * k]] = -(1 << 62)
    off[E] = 1 << 62
    if E > 8:
        off[E // 2] = min(M, int(off[E // 2 - 1]) + M // 8)
    return off


@pytest.mark.parametrize("M,E,d", [(700, 3, 1096), (1500, 4, 4096), (4396, 3, 4096), (3000, 70, 1032), (18000, 70, 520),
                                   (9000, 200, 520)])
def test_bad_offsets_in_tiles(ops, M, E, d):  # noqa: F811
    """Whatever the offsets hold, rows count as the definition says and no other row is touched."""
    n, t = 40, torch.bfloat16
    X, dY = randn(1, (M, n), 1.0, t).cuda(), randn(2, (M, d), 0.1, t).cuda()
    W = randn(3, (E, d, n), 0.05, t).cuda()
    (xq, sx), q = ops.fp8_quant_act(torch.nn.functional.pad(X, (0, 8))), ops.fp8_quant_weight(torch.nn.functional.pad(W, (0, 8)))
    x, dy, w = X.double(), dY.double(), W.double()
    x8, w8 = values(xq, sx, 1), [values(q["wq"][e], q["sw"][e], 128) for e in range(E)]
    for seed in (1, 2):
        off = _wild_offsets(seed, E, M)
        b = ref.boundaries(off, M)
        o = torch.from_numpy(off).cuda()
        if seed == 2:  # rows in front of the first group and behind the last
            b = ref.boundaries([50, *(off[1:-1] // 2), off[-2] // 2], M)
            o = torch.tensor([50, *(off[1:-1] // 2), off[-2] // 2], device="cuda")
        outs = [torch.full((M, c), 7.0, dtype=t, device="cuda") for c in (d, n, n, d, d)]
        Wt = W.transpose(1, 2).contiguous()
        ops.grouped_linear(X, o, W, out=outs[0])
        ops.grouped_linear(dY, o, Wt, out=outs[1])
        ops.grouped_linear_dx(dY, o, W, out=outs[2])
        ops.grouped_linear_dx(X, o, Wt, out=outs[3])
        ops.fp8_grouped_linear(xq, sx, o, q["wq"], q["sw"], out=outs[4])
        dW = ops.grouped_linear_dw(dY, X, o, dtype=torch.float32)
        for out in outs:
            assert (out[:b[0]] == 7).all() and (out[b[-1]:] == 7).all()
        for e in range(E):
            r = slice(b[e], b[e + 1])
            we, wt = w[e], w[e].t().contiguous()
            for out, a, c, k in zip(outs, (x, dy, dy, x), (we, wt, wt, we), (n, d, d, n)):
                check(out[r], a[r], c, k, f"group {e}")
            check(outs[4][r], x8[r], w8[e], 48, f"8 bits, group {e}", True)
            check(dW[e], dy[r].t().contiguous(), x[r].t().contiguous(), b[e + 1] - b[e], f"dW {e}")
