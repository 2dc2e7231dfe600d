"""Sizes of the adapters' forward call where the gradients' transposes would be more tiles than a
grid holds: the forward transposes nothing and takes them (first part on the CPU, where nothing
reaches a device)."""
import pytest
import torch

from integer_rank_adaptation_amd import binding as B

P = [0x1000000 * (i + 1) for i in range(8)]  # 16-byte aligned, never dereferenced


@pytest.mark.parametrize("M", [40, 1000])
@pytest.mark.parametrize("L,d,n,r", [(4096, 1 << 17, 1 << 17, 1), (4096, 1 << 17, 1 << 17, 64), (2048, 1 << 18, 1 << 18, 20),
                                     (4096, 1 << 16, 1 << 16, 65)])
def test_forward_takes_wide_factors(M, L, d, n, r):
    lib = B.lib()
    assert lib.intlora_adapters_ws_bytes(M, L, d, n, r, 0) > 0
    # a workspace of 16 bytes: EWORKSPACE where the sizes are taken
    assert lib.intlora_adapters_fwd(M, L, d, n, r, 0, P[0], P[1], P[2], P[3], P[4], P[5], P[6], P[7], 16,
                                    None) == B.INTLORA_EWORKSPACE
    assert lib.intlora_adapters_ws_bytes(M, L, d, n, r, 1) == 0
    assert lib.intlora_adapters_grad(M, L, d, n, r, 0, 2, P[0], P[1], P[2], P[3], P[4], P[5], None, None, P[6], P[7],
                                     P[7], 16, None) == B.INTLORA_ESHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("M", [40, 700])
def test_wide_factors(M):
    """4096 adapters of rank 1 over 2^17 columns on both sides, few rows and listed ones.  All
    inputs are small whole numbers, so every sum is exact in binary32 and a row has one value, up
    to the one rounding to bf16: |h| <= 2^15 has 15 bits (two bf16 pieces hold 16), |base + 2 A h|
    < 2^20."""
    from integer_rank_adaptation_amd import ops

    L, w = 4096, 1 << 17
    g = torch.Generator(device="cuda").manual_seed(M)
    ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    x, A, Bm, base = ints(-1, 1, M, w), ints(-8, 8, L, w, 1), ints(-1, 1, L, 1, w), ints(-100, 100, M, w)
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    ids[:4] = torch.tensor([0, L - 1, L - 1, -1], dtype=torch.int32)
    y = ops.adapters_linear(base, x, ids, A, Bm, torch.full((L,), 2.0, device="cuda"))
    for t in range(M):
        a = int(ids[t])
        want = base[t].double()
        if a >= 0:
            h = (x[t].double() * Bm[a, 0].double()).sum()
            assert abs(h) <= 1 << 15
            want = want + 2 * h * A[a, :, 0].double()
        assert torch.equal(y[t], want.to(torch.bfloat16)), t
