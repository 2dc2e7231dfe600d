"""The floating-point layers at sizes past one launch's grid (2^32 work-items) on the GPU."""
import numpy as np
import pytest
import torch

from oracle import fplinear as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from integer_rank_adaptation_amd import ops as _ops

    _ops.B.lib()
    return _ops


def randn(seed, shape, std=1.0, dtype=torch.bfloat16):
    g = np.random.Generator(np.random.PCG64(seed))
    return torch.from_numpy((g.standard_normal(shape) * std).astype(np.float32)).to(dtype)


def test_quantizer_of_more_rows_than_one_grid(ops):
    """2^28 rows and more of 16 columns: zeros but for rows at both ends and about the 2^28th."""
    M, n = (1 << 28) + 1000, 16
    X = torch.zeros((M, n), dtype=torch.bfloat16, device="cuda")
    live = [(0, 40), ((1 << 28) - 40, (1 << 28) + 40), (M - 40, M)]
    want = {}
    for i, (a, b) in enumerate(live):
        x = randn(i, (b - a, n), 3.0)
        X[a:b] = x.cuda()
        want[a, b] = ref.quantize(x.double().numpy(), 1)
    xq = torch.full((M, n), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sx = torch.zeros((M, ops.fp8_scale_bytes(n)), dtype=torch.uint8, device="cuda")
    ops.fp8_quant_act(X, out=(xq, sx))
    codes = xq.view(torch.uint8)
    for (a, b), (cq, cs) in want.items():
        assert np.array_equal(codes[a:b].cpu().numpy(), cq) and np.array_equal(sx[a:b].cpu().numpy(), cs)
    for (_, a), (b, _) in zip(live, live[1:]):
        assert int(codes[a:b].max()) == 0
        assert int(sx[a:b].min()) == 127 and int(sx[a:b].max()) == 127


def test_more_small_tiles_than_one_grid(ops):
    """4096 groups that average one row, of 520448 columns: tiles of 128 x 128 would be more than
    2^24 blocks of 256 threads.  Three groups have rows; the input gradient (short contraction)
    and the forward product on the same weights read the other way round."""
    E, n, d = 4096, 520448, 8
    rows = {0: 3, 2000: 290, 4095: 3803}
    M = sum(rows.values())
    off, at = torch.zeros(E + 1, dtype=torch.int64), 0
    for e in range(E):
        at += rows.get(e, 0)
        off[e + 1] = at
    assert (M // 128 + E - 1) * (n // 128) >= 1 << 24
    W = torch.zeros((E, d, n), dtype=torch.bfloat16, device="cuda")
    for e in rows:
        W[e] = randn(e, (d, n), 0.05).cuda()
    dY = randn(7, (M, d))
    offd = off.cuda()
    cols = np.unique(np.concatenate([np.arange(300), n // 2 + np.arange(-130, 130), n - 1 - np.arange(300)]))
    pick = torch.from_numpy(cols).cuda()
    dX = ops.grouped_linear_dx(dY.cuda(), offd, W)
    Y = ops.grouped_linear(dY.cuda(), offd, W.view(E, n, d))
    for e in rows:
        a, b = int(off[e]), int(off[e + 1])
        g = dY[a:b].double().numpy()
        for out, w in ((dX, W[e][:, pick]), (Y, W.view(E, n, d)[e][pick].t())):
            w = w.cpu().double().numpy()
            want, mag = g @ w, np.abs(g) @ np.abs(w)
            acc = (d + 16) * 2.0**-23 * mag  # d terms in binary32, any order; then one rounding to bf16
            got = out[a:b][:, pick].cpu().double().numpy()
            assert (np.abs(got - want) <= acc + 2.0**-8 * (np.abs(want) + acc)).all()
