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
