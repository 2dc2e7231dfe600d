"""Host side of the floating-point layers and of gradient clipping (CPU): refusals of the C
entry points (nothing reaches a device), argument checks of the tensor calls, and the plain
definitions the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

from integer_rank_adaptation_amd import binding as B
from integer_rank_adaptation_amd import ops
from oracle import fplinear as ref

FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call below ends in validation
OK, EINVAL, ESHAPE, EALIGN, EWS = (B.INTLORA_OK, B.INTLORA_EINVAL, B.INTLORA_ESHAPE, B.INTLORA_EALIGN,
                                   B.INTLORA_EWORKSPACE)


@pytest.fixture(scope="module")
def lib():
    return B.lib()


@pytest.mark.parametrize("args,expect", [
    ((4, 64, 3, FAKE, FAKE, FAKE), EINVAL),              # no such type
    ((4, 24, 0, FAKE, FAKE, FAKE), ESHAPE),              # n not a multiple of 16
    ((-1, 64, 0, FAKE, FAKE, FAKE), ESHAPE),
    ((4, 0, 0, FAKE, FAKE, FAKE), ESHAPE),
    ((4, (1 << 20) + 16, 0, FAKE, FAKE, FAKE), ESHAPE),
    ((1 << 31, 64, 0, FAKE, FAKE, FAKE), ESHAPE),
    ((4, 64, 2, None, FAKE, FAKE), EINVAL),
    ((4, 64, 1, FAKE, FAKE + 8, FAKE), EALIGN),
    ((0, 64, 0, None, None, None), OK),
])
def test_quant_act_refusals(lib, args, expect):
    assert lib.intlora_fp8_quant_act(*args, None) == expect
    assert bool(lib.intlora_last_error()) == (expect != OK)


@pytest.mark.parametrize("args,expect", [
    ((1, 64, 64, 5, FAKE, FAKE, FAKE, None, None), EINVAL),
    ((0, 64, 64, 0, FAKE, FAKE, FAKE, None, None), ESHAPE),
    ((4097, 64, 64, 0, FAKE, FAKE, FAKE, None, None), ESHAPE),
    ((1, 64, 40, 0, FAKE, FAKE, FAKE, None, None), ESHAPE),
    ((1, 64, 64, 0, FAKE, FAKE, FAKE, FAKE, None), EINVAL),  # the transposed pair: both or neither
    ((1, 64, 64, 0, FAKE, FAKE, FAKE, None, FAKE), EINVAL),
    ((1, 40, 64, 0, FAKE, FAKE, FAKE, FAKE, FAKE), ESHAPE),  # transposed rows of 40 codes
    ((1, 64, 64, 0, FAKE, None, FAKE, None, None), EINVAL),
    ((1, 64, 64, 0, FAKE, FAKE, FAKE + 4, None, None), EALIGN),
    ((1, 64, 64, 0, FAKE, FAKE, FAKE, FAKE + 2, FAKE), EALIGN),
    ((1, 0, 64, 0, None, None, None, None, None), OK),
])
def test_quant_weight_refusals(lib, args, expect):
    assert lib.intlora_fp8_quant_weight(*args, None) == expect


@pytest.mark.parametrize("args,expect", [
    ((4, 8, 24, FAKE, FAKE, FAKE, FAKE, FAKE), ESHAPE),
    ((-1, 8, 32, FAKE, FAKE, FAKE, FAKE, FAKE), ESHAPE),
    ((4, (1 << 20) + 1, 32, FAKE, FAKE, FAKE, FAKE, FAKE), ESHAPE),
    ((1 << 30, 1 << 20, 32, FAKE, FAKE, FAKE, FAKE, FAKE), ESHAPE),  # more tiles than a grid holds
    ((4, 8, 32, FAKE, None, FAKE, FAKE, FAKE), EINVAL),
    ((4, 8, 32, FAKE, FAKE, FAKE, FAKE, FAKE + 2), EALIGN),
    ((0, 8, 32, None, None, None, None, None), OK),
    ((4, 0, 32, None, None, None, None, None), OK),
])
def test_fp8_linear_refusals(lib, args, expect):
    assert lib.intlora_fp8_linear_fwd(*args, None) == expect
    M, d, n, xq, sx, wq, sw, y = args
    assert lib.intlora_fp8_grouped_linear_fwd(M, 3, d, n, xq, sx, FAKE, wq, sw, y, None) == expect


def test_grouped_refusals(lib):
    fwd, dx, dw = lib.intlora_grouped_linear_fwd, lib.intlora_grouped_linear_dx, lib.intlora_grouped_linear_dw
    for f in (fwd, dx):
        good = [8, 2, 16, 16, 0, FAKE, FAKE, FAKE, FAKE, None]

        def call(**kw):
            a = list(good)
            for k, v in kw.items():
                a[int(k[1:])] = v
            return f(*a)

        assert call(a4=2) == EINVAL          # fp32 operands
        assert call(a1=0) == ESHAPE and call(a1=4097) == ESHAPE
        assert call(a2=12) == ESHAPE and call(a3=20) == ESHAPE
        assert call(a0=-1) == ESHAPE
        assert call(a6=None) == EINVAL       # several groups need offsets
        assert call(a6=FAKE + 8) == EALIGN
        assert call(a5=None) == EINVAL and call(a7=FAKE + 4) == EALIGN and call(a8=None) == EINVAL
        assert call(a0=0) == OK
    assert fwd(8, 2, 0, 16, 0, FAKE, FAKE, FAKE, FAKE, None) == OK
    assert dx(8, 2, 0, 16, 0, FAKE, FAKE, FAKE, FAKE, None) == ESHAPE  # a product over nothing
    assert dw(8, 2, 16, 16, 0, 1, FAKE, FAKE, FAKE, FAKE, None) == EINVAL  # bf16 in, fp16 out
    assert dw(8, 2, 16, 16, 2, 2, FAKE, FAKE, FAKE, FAKE, None) == EINVAL
    assert dw(8, 2, 16, 16, 0, 2, FAKE, FAKE, FAKE, FAKE + 2, None) == EALIGN
    assert dw(8, 2, 0, 16, 0, 2, FAKE, FAKE, FAKE, FAKE, None) == OK
    assert fwd(8, 1, 16, 16, 0, FAKE, None, FAKE, None, None) == EINVAL  # one group may do without offsets
    assert lib.intlora_fp8_grouped_linear_fwd(8, 2, 16, 16, FAKE, FAKE, None, FAKE, FAKE, FAKE, None) == EINVAL


def _arrays(ptrs, numel, types):
    k = len(numel)
    return (ctypes.c_void_p * k)(*ptrs), (ctypes.c_int64 * k)(*numel), (ctypes.c_int32 * k)(*types)


def test_grad_refusals(lib):
    p, n, t = _arrays([FAKE, 2 * FAKE], [100, 40000], [2, 0])
    assert lib.intlora_grad_ws_bytes(2, n) == (1 + 3) * 8
    assert lib.intlora_grad_ws_bytes(0, None) == 16
    s = lib.intlora_grad_sumsq
    assert s(2, p, n, t, FAKE, FAKE, 31, None) == EWS
    assert s(2, p, n, t, FAKE, None, 32, None) == EWS
    assert s(2, p, n, t, None, FAKE, 32, None) == EINVAL
    assert s(2, None, n, t, FAKE, FAKE, 32, None) == EINVAL
    assert s(-1, p, n, t, FAKE, FAKE, 32, None) == ESHAPE
    assert s(65537, p, n, t, FAKE, FAKE, 32, None) == ESHAPE
    bad = _arrays([FAKE, 2 * FAKE], [100, -1], [2, 0])
    assert s(2, *bad, FAKE, FAKE, 1 << 20, None) == ESHAPE
    bad = _arrays([FAKE, 2 * FAKE], [100, 5], [2, 3])
    assert s(2, *bad, FAKE, FAKE, 1 << 20, None) == EINVAL
    bad = _arrays([FAKE, 2 * FAKE + 8], [100, 5], [2, 0])
    assert s(2, *bad, FAKE, FAKE, 1 << 20, None) == EALIGN
    bad = _arrays([FAKE, None], [100, 5], [2, 0])
    assert s(2, *bad, FAKE, FAKE, 1 << 20, None) == EINVAL


def _clip(lib, grads, outs, numel, types, max_norm=1.0, sumsq=FAKE):
    p, n, t = _arrays(grads, numel, types)
    return lib.intlora_grad_clip(len(numel), p, (ctypes.c_void_p * len(numel))(*outs), n, t, sumsq, max_norm, None, None)


def test_clip_refusals(lib):
    a, b = 0x100000, 0x200000
    assert _clip(lib, [a], [a], [10], [2], max_norm=-1.0) == EINVAL
    assert _clip(lib, [a], [a], [10], [2], max_norm=math.nan) == EINVAL
    assert _clip(lib, [a], [a], [10], [2], sumsq=None) == EINVAL
    assert _clip(lib, [a], [None], [10], [2]) == EINVAL
    assert _clip(lib, [a], [b + 4], [10], [2]) == EALIGN
    # overlaps: the same output twice, the same gradient twice in place, an output inside
    # another tensor's input, a shifted output, an output read by a later entry
    assert _clip(lib, [a, b], [b, b], [10, 10], [2, 2]) == EINVAL
    assert _clip(lib, [a, a], [a, a], [10, 10], [2, 2]) == EINVAL
    assert _clip(lib, [a, b], [b + 16, 0x300000], [10, 10], [2, 2]) == EINVAL
    assert _clip(lib, [a], [a + 16], [100], [2]) == EINVAL
    assert _clip(lib, [a + 16], [a], [100], [2]) == EINVAL
    assert _clip(lib, [a, a], [a, b], [10, 10], [2, 2]) == EINVAL
    assert b"overlaps" in lib.intlora_last_error()


def test_outputs_may_not_overlap(lib):
    x, s, w, v, y, off = (0x1000000 * k for k in range(1, 7))
    M, E, d, n = 8, 2, 32, 64
    # (one byte of overlap at either end is out of reach: pointers are multiples of 16)
    for bad in (x, x + M * n - 16, x - 16, s, w + E * d * n - 16, v, off):
        assert lib.intlora_fp8_grouped_linear_fwd(M, E, d, n, x, s, off, w, v, bad, None) == EINVAL
    for bad in (x, w + d * n - 16):
        assert lib.intlora_fp8_linear_fwd(M, d, n, x, s, w, v, bad, None) == EINVAL
    for f, rows, cols in ((lib.intlora_grouped_linear_fwd, n, d), (lib.intlora_grouped_linear_dx, d, n)):
        for bad in (x, x + 2 * M * rows - 16, x - 2 * M * cols + 16, w + 2 * E * d * n - 16, off):
            assert f(M, E, d, n, 0, x, off, w, bad, None) == EINVAL
    dw = lib.intlora_grouped_linear_dw
    for bad in (x, w + 2 * M * n - 16, w - 4 * E * d * n + 16):
        assert dw(M, E, d, n, 0, 2, x, w, off, bad, None) == EINVAL
    assert b"overlaps" in lib.intlora_last_error()
    assert lib.intlora_fp8_quant_act(M, n, 0, x, x, s, None) == EINVAL
    assert lib.intlora_fp8_quant_act(M, n, 0, x, y, x + 2 * M * n - 16, None) == EINVAL
    assert lib.intlora_fp8_quant_act(M, n, 2, x, y, x + 4 * M * n - 16, None) == EINVAL
    assert lib.intlora_fp8_quant_act(M, n, 0, x, y, y + 16, None) == EINVAL
    for wq, sw, wt, st in ((x, s, None, None), (w, x, None, None), (w, s, w, v), (w, s, v, s), (w, s, v, x + 16)):
        assert lib.intlora_fp8_quant_weight(E, d, n, 0, x, wq, sw, wt, st, None) == EINVAL


def test_clip_sum_and_norm_may_not_overlap(lib):
    def call(sumsq, norm, grads=(0x100000, 0x200000), out=(0x300000, 0x400000)):
        k, numel = len(grads), (ctypes.c_int64 * 2)(64, 64)
        g, o, t = (ctypes.c_void_p * k)(*grads), (ctypes.c_void_p * k)(*out), (ctypes.c_int32 * 2)(2, 0)
        return lib.intlora_grad_clip(k, g, o, numel, t, sumsq, 1.0, norm, None)

    assert call(0x500000, 0x500000) == EINVAL             # the sum itself
    assert call(0x300000 + 240, 0x500000) == EINVAL       # a sum that a block overwrites
    assert call(0x500000, 0x400000) == EINVAL             # a norm inside an output
    assert call(0x500000, 0x200000 + 112) == EINVAL       # ... inside an input
    assert b"overlaps" in lib.intlora_last_error()
    assert call(0x100000, 0x600000, out=(0x100000, 0x200000)) == EINVAL  # in place


def test_tensor_calls_refuse_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64)
    for call in (lambda: ops.fp8_quant_act(x), lambda: ops.fp8_quant_weight(x), lambda: ops.fp8_quant_act(x[0]),
                 lambda: ops.grouped_linear(x, None, x[None]), lambda: ops.grouped_linear_dx(x, None, x[None]),
                 lambda: ops.grouped_linear_dw(x, x, None), lambda: ops.fp8_linear(x, x, x, x)):
        with pytest.raises((ValueError, RuntimeError)):
            call()


# ------------------------------------------------------------------ the definitions themselves
def test_e4m3_table_and_rounding_agree_with_torch():
    v = ref.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    x = np.random.Generator(np.random.PCG64(1)).standard_normal(200000) * 60
    x = np.concatenate([x[np.abs(x) <= 448], v[np.isfinite(v)], [447.9, 464.0 - 1e-9, 2.0**-10, 3 * 2.0**-10]]).astype(np.float32)
    want = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.to_e4m3(x), want)


def test_scale_exponent_is_the_least():
    g = np.random.Generator(np.random.PCG64(2))
    vals = [448.0, np.nextafter(np.float32(448), np.float32(999)), 1.75, 1.7500001, 1e-45, 2.0**-118, 3.4028234e38]
    for a in [float(np.float32(x)) for x in vals] + [float(np.float32(x)) for x in np.exp(g.uniform(-80, 88, 500))]:
        e = ref.scale_exponent(a)
        assert math.ldexp(a, -e) <= 448 and (e == -127 or math.ldexp(a, 1 - e) > 448)
    assert ref.scale_exponent(0.0) == 0


def test_quantize_error_is_half_a_step():
    """Every value is within half an e4m3 step of its code: 2^-4 of it, or half of 2^(e - 9)."""
    x = np.random.Generator(np.random.PCG64(3)).standard_normal((9, 400)).astype(np.float32)
    for rows in (1, 128):
        c, s = ref.quantize(x, rows)
        d = ref.dequantize(c, s, rows)
        step = np.exp2(np.repeat(np.repeat(s.astype(float) - 127, rows, 0)[:9], 128, 1)[:, :400] - 10)
        assert (np.abs(d - x) <= np.maximum(np.abs(x) * 2.0**-4, step)).all()
        assert s.shape == (-(-9 // rows), 4) and (s[:, -(-400 // 128):] == 127).all()


def test_boundaries():
    assert ref.boundaries([0, 3, 3, 8], 8) == [0, 3, 3, 8]
    assert ref.boundaries([-4, 5, 2, 99], 8) == [0, 5, 5, 8]
