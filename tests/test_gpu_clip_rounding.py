"""The scaled gradients bit for bit: the binary32 product with the binary32 factor, rounded once
more for 16-bit gradients."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("sumsq,max_norm", [(9.0, 1.0), (2.0, 1.2345), (1e6, 0.7), (0.3, 0.5), (1e60, 1.0), (0.01, 0.1)])
def test_every_value_is_rounded_as_stated(dtype, sumsq, max_norm):
    from integer_rank_adaptation_amd import ops

    if dtype == torch.float32:
        bits = np.random.Generator(np.random.PCG64(1)).integers(0, 1 << 32, 100_000, dtype=np.uint32)
        g = torch.from_numpy(bits.view(np.float32).copy())
    else:
        g = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(dtype)
    c = np.float32(min(1.0, max_norm / (np.sqrt(np.float64(sumsq)) + 1e-6)))
    want = (g.float() * torch.tensor(c)).to(dtype)  # (CPU)
    out = torch.zeros_like(g, device="cuda")
    norm = ops.grad_clip([g.cuda()], torch.tensor([sumsq], dtype=torch.float64, device="cuda"), max_norm, out=[out])
    assert np.float32(norm.item()) == np.float32(np.sqrt(np.float64(sumsq)))
    got = out.cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    ints = torch.int32 if dtype == torch.float32 else torch.int16
    assert torch.equal(got.view(ints)[~nan], want.view(ints)[~nan])
