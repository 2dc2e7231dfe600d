"""Sizes of the calls that restore saved codes (CPU; nothing reaches a device): the restoring counts
its units of 16 codes in 32 bits, and both calls refuse what does not fit."""
import pytest

from integer_rank_adaptation_amd import binding as B

P = [0x1000000 * (i + 1) for i in range(6)]  # 16-byte aligned, never dereferenced
# (rows, columns): units at and past 2^32 - 256, and the last size before it
PAST = [(65536, 1 << 20), (65552, 1 << 20), (70000, 1 << 20), (9_000_000, 8192), (1 << 28, 256), ((1 << 28) - 16, 256),
        ((1 << 30), 64)]
BELOW = [(65535, 1 << 20), ((1 << 28) - 17, 256)]


def dw(M, n):
    # a workspace of 512 bytes: EWORKSPACE where the sizes are taken
    return B.lib().intlora_grouped_linear_dw_fp8(M, 1, 8, n, 0, 2, P[0], P[1], P[2], None, P[4], P[5], 512, None)


def restore(M, n):
    # no codes: EINVAL where the sizes are taken
    return B.lib().intlora_fp8_dequant_act(M, n, 0, None, P[1], P[2], None)


@pytest.mark.parametrize("M,n", PAST)
def test_past_the_count(M, n):
    assert dw(M, n) == B.INTLORA_ESHAPE and "2^36 - 2^12" in B.lib().intlora_last_error().decode()
    assert restore(M, n) == B.INTLORA_ESHAPE


@pytest.mark.parametrize("M,n", BELOW)
def test_below_the_count(M, n):
    assert dw(M, n) == B.INTLORA_EWORKSPACE
    assert restore(M, n) == B.INTLORA_EINVAL
