"""Adapters of many requests on the GPU against the plain definition in binary64."""
import numpy as np
import pytest
import torch

from oracle import adapters as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def ops():
    from integer_rank_adaptation_amd import ops

    return ops


def make(M, L, d, n, r, x="bf16", kind="random", seed=0):
    g = torch.Generator().manual_seed(seed * 1000003 + M * 131 + r)
    t = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(DT[x])
    if kind == "runs":
        ids = torch.sort(torch.randint(-1, L, (M,), generator=g, dtype=torch.int32)).values
    elif kind == "one":
        ids = torch.full((M,), L - 1, dtype=torch.int32)
    elif kind == "none":
        ids = torch.full((M,), -1, dtype=torch.int32)
    else:
        ids = torch.randint(0, L, (M,), generator=g, dtype=torch.int32)
        ids[torch.rand(M, generator=g) < 0.15] = -1
    return dict(base=t(M, d), x=t(M, n), index=ids, A=t(L, d, r, std=0.2), B=t(L, r, n, std=n ** -0.5),
                scale=torch.rand(L, generator=g) * 2 - 0.5, dy=t(M, d, std=0.1), dxb=t(M, n, std=0.1))


def dev(c):
    return {k: v.cuda() for k, v in c.items()}


def f64(t):
    return t.double().cpu().numpy()


def half_step(v, dtype):
    """Half a step of the type around v: eps / 2 of it, and of the smallest normal number."""
    f = torch.finfo(dtype)
    return f.eps / 2 * np.maximum(np.abs(v), f.tiny)


def check(got, want, spread, what):
    err = np.abs(f64(got) - want)
    # the rounding of what lies at most `spread` from `want`
    tol = spread + half_step(np.abs(want) + spread, got.dtype)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / np.maximum(tol, 1e-300)):.3g}"


def forward(ops, c, base=True):
    g = dev(c)
    y = ops.adapters_linear(g["base"] if base else None, g["x"], g["index"], g["A"], g["B"], g["scale"])
    want, spread = ref.forward(f64(c["base"]) if base else None, f64(c["x"]), c["index"].numpy(), f64(c["A"]),
                               f64(c["B"]), f64(c["scale"]))
    check(y, want, spread, "y")
    return g, y


def backward(ops, c, dtype=torch.float32, base=True):
    g = dev(c)
    dx, dA, dB = ops.adapters_linear_grad(g["dy"], g["x"], g["index"], g["A"], g["B"], g["scale"],
                                          base=g["dxb"] if base else None, dtype=dtype)
    want, tol = ref.backward(f64(c["dxb"]) if base else None, f64(c["dy"]), f64(c["x"]), c["index"].numpy(),
                             f64(c["A"]), f64(c["B"]), f64(c["scale"]))
    assert dA.dtype == dB.dtype == dtype
    for k, v in (("dx", dx), ("dA", dA), ("dB", dB)):
        check(v, want[k], tol[k], k)
    return g, (dx, dA, dB)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 100, 256, 257, 640, 641, 1025, 1500])
@pytest.mark.parametrize("x,r,d,n", [("bf16", 16, 72, 136), ("fp16", 20, 136, 72), ("bf16", 3, 64, 1096),
                                     ("fp16", 16, 264, 4096), ("bf16", 13, 520, 4104), ("fp16", 128, 1000, 2048)])
@pytest.mark.parametrize("L", [5, 200])
def test_rows(ops, M, x, r, d, n, L):
    forward(ops, make(M, L, d, n, r, x))


@pytest.mark.parametrize("M,L,d,n,r,x,kind", [
    (33, 1, 8192, 4096, 64, "bf16", "one"), (40, 1, 8192, 4096, 64, "bf16", "one"),
    (25, 2, 14336, 4104, 100, "fp16", "random"), (31, 2, 14344, 4104, 101, "fp16", "random"),
    (200, 8, 4096, 4096, 16, "bf16", "runs"), (230, 8, 4096, 4096, 16, "bf16", "runs"),
    (150, 40, 4104, 2056, 64, "fp16", "random"), (260, 40, 4104, 2056, 64, "fp16", "random"),
    (640, 2, 1032, 776, 20, "bf16", "random"), (640, 2, 2056, 1032, 20, "bf16", "random"),
])
def test_around_the_lists(ops, M, L, d, n, r, x, kind):
    """Either side of where rows are listed first, which depends on rows, adapters, sizes and rank."""
    forward(ops, make(M, L, d, n, r, x, kind))


@pytest.mark.parametrize("r", [1, 2, 7, 8, 15, 17, 24, 32, 33, 48, 63, 64, 65, 100, 127, 128])
@pytest.mark.parametrize("x,M", [("bf16", 37), ("fp16", 37), ("bf16", 1100), ("fp16", 300)])
def test_ranks(ops, r, x, M):
    forward(ops, make(M, 3, 104, 200, r, x, "runs"))


@pytest.mark.parametrize("d,n", [(8, 8), (8, 520), (520, 8), (64, 64), (72, 264), (1032, 2056), (56, 5000)])
@pytest.mark.parametrize("M", [5, 1030])
def test_sizes(ops, d, n, M):
    forward(ops, make(M, 4, d, n, 12, "bf16", "runs"))
    forward(ops, make(M, 4, d, n, 8, "fp16", "random"), base=False)


@pytest.mark.parametrize("kind", ["runs", "one", "none", "random"])
@pytest.mark.parametrize("M,L", [(40, 1), (40, 64), (2000, 40)])
def test_index(ops, kind, M, L):
    forward(ops, make(M, L, 80, 96, 16, "bf16", kind))
    forward(ops, make(M, L, 80, 96, 16, "bf16", kind), base=False)


def test_index_outside(ops):
    c = make(50, 3, 64, 64, 8)
    c["index"][:6] = torch.tensor([3, 4, 1 << 30, -2, -(1 << 31), (1 << 31) - 1], dtype=torch.int32)
    _, y = forward(ops, c)
    assert torch.equal(y[:6].cpu(), c["base"][:6])


@pytest.mark.parametrize("M", [33, 1200])
def test_in_place(ops, M):
    """In place the same values; rows without an adapter keep their bits, NaN payloads too."""
    c = make(M, 4, 136, 72, 16)
    bare = c["index"] < 0
    c["base"].view(torch.int16)[bare] = torch.arange(0, 136, dtype=torch.int16) + 0x7F81  # NaN of many payloads
    g = dev(c)
    y = ops.adapters_linear(g["base"], g["x"], g["index"], g["A"], g["B"], g["scale"])
    z = ops.adapters_linear(g["base"], g["x"], g["index"], g["A"], g["B"], g["scale"], out=g["base"])
    assert z is g["base"] and torch.equal(y.view(torch.int16), z.view(torch.int16))
    assert torch.equal(z.view(torch.int16)[bare.cuda()].cpu(), c["base"].view(torch.int16)[bare])


@pytest.mark.parametrize("M", [48, 1100])
@pytest.mark.parametrize("x", ["bf16", "fp16"])
def test_non_finite(ops, M, x):
    """A NaN or an infinity stays in its row (tokens) or with its adapter (factors)."""
    c = make(M, 4, 64, 96, 5, x)
    clean = ops.adapters_linear(*[dev(c)[k] for k in ("base", "x", "index", "A", "B", "scale")])
    c["index"][:4] = torch.tensor([0, 1, 2, 1], dtype=torch.int32)
    clean = ops.adapters_linear(*[dev(c)[k] for k in ("base", "x", "index", "A", "B", "scale")])
    c["x"][0, 3] = float("nan")
    c["A"][2, 7, 1] = float("inf")
    c["B"][3, 4, 50] = float("-inf")
    y = ops.adapters_linear(*[dev(c)[k] for k in ("base", "x", "index", "A", "B", "scale")])
    ids = c["index"].cuda()
    assert y[0].isnan().all()
    untouched = ((ids < 2) & (torch.arange(M, device="cuda") > 0))
    assert torch.equal(y[untouched], clean[untouched])
    two = ids == 2
    two_cols = torch.arange(64, device="cuda") != 7
    assert torch.equal(y[two][:, two_cols], clean[two][:, two_cols]) and not y[two][:, 7].isfinite().any()
    assert not y[ids == 3].isfinite().any()


@pytest.mark.parametrize("x,big", [("fp16", 6e4), ("bf16", 1e30)])
def test_wide_range(ops, x, big):
    """Low-rank terms far outside fp16's range, and next to nothing."""
    c = make(40, 3, 64, 128, 8, x)
    c["x"][:10] *= big / 8
    c["A"] *= 1e-3 if x == "fp16" else 1.0
    c["x"][10:20] *= 1e-4
    c["x"].clamp_(-big, big)
    forward(ops, c)


@pytest.mark.parametrize("M,L,d,n,r,x,kind", [
    (1, 1, 8, 8, 1, "bf16", "one"), (31, 3, 72, 136, 4, "bf16", "random"), (32, 2, 64, 64, 16, "fp16", "runs"),
    (33, 2, 136, 72, 17, "bf16", "one"), (300, 7, 72, 200, 20, "fp16", "random"), (700, 2, 264, 64, 64, "bf16", "runs"),
    (700, 2, 64, 264, 33, "fp16", "runs"), (1500, 3, 136, 72, 128, "bf16", "random"),
    (1500, 40, 72, 136, 100, "fp16", "random"), (2100, 5, 640, 72, 20, "fp16", "runs"),
    (1100, 3, 72, 1096, 7, "bf16", "none"), (256, 2, 64, 2056, 16, "bf16", "runs"), (257, 2, 2056, 64, 16, "bf16", "runs"),
    (600, 200, 64, 72, 8, "fp16", "random"), (2000, 300, 264, 136, 9, "bf16", "runs"),
    (64, 3, 1096, 264, 20, "fp16", "random"), (65, 3, 1096, 264, 20, "fp16", "random"), (70, 2, 2056, 1032, 64, "bf16", "runs"),
    (100, 80, 72, 136, 17, "bf16", "random"), (250, 5, 136, 72, 128, "fp16", "one"),
])
def test_gradients(ops, M, L, d, n, r, x, kind):
    c = make(M, L, d, n, r, x, kind)
    backward(ops, c)
    backward(ops, c, dtype=DT[x], base=False)


def test_gradients_without_rows(ops):
    c = make(4, 2, 16, 24, 3)
    g = dev({k: (v[:0] if k in ("base", "x", "index", "dy", "dxb") else v) for k, v in c.items()})
    y = ops.adapters_linear(g["base"], g["x"], g["index"], g["A"], g["B"], g["scale"])
    dA, dB = torch.full((2, 16, 3), 7.0, device="cuda"), torch.full((2, 3, 24), 7.0, device="cuda")
    dx, a, b = ops.adapters_linear_grad(g["dy"], g["x"], g["index"], g["A"], g["B"], g["scale"],
                                        out=(None, dA, dB))
    assert y.shape == (0, 16) and dx.shape == (0, 24) and a is dA and not dA.any() and not dB.any()


def test_gradients_in_place_and_without_dx(ops):
    c = make(200, 4, 64, 72, 8, kind="runs")
    g, (dx, dA, dB) = backward(ops, c)
    o = ops.adapters_linear_grad(g["dy"], g["x"], g["index"], g["A"], g["B"], g["scale"], dtype=torch.float32,
                                 need_dx=False)
    assert o[0] is None and torch.equal(o[1], dA) and torch.equal(o[2], dB)
    o = ops.adapters_linear_grad(g["dy"], g["x"], g["index"], g["A"], g["B"], g["scale"], base=g["dxb"],
                                 out=(g["dxb"], torch.empty_like(dA), torch.empty_like(dB)))
    assert o[0] is g["dxb"] and torch.equal(o[0], dx) and torch.equal(o[1], dA) and torch.equal(o[2], dB)


def test_gradients_non_finite(ops):
    """A NaN token reaches its own dX row and its adapter's factors only."""
    c = make(100, 3, 64, 72, 8)
    c["index"][:] = torch.arange(100) % 3
    g, (dx, dA, dB) = backward(ops, c)
    g["x"][3, 5] = float("nan")  # adapter 0
    x2, a2, b2 = ops.adapters_linear_grad(g["dy"], g["x"], g["index"], g["A"], g["B"], g["scale"], base=g["dxb"],
                                          dtype=torch.float32)
    assert torch.equal(x2, dx) and torch.equal(a2[1:], dA[1:]) and torch.equal(b2[1:], dB[1:])
    assert a2[0].isnan().all() and b2[0, :, 5].isnan().all()
    assert torch.equal(b2[0, :, :5], dB[0, :, :5])
    g["x"][3, 5] = 0
    g["dy"][4, 0] = float("inf")  # adapter 1
    x3, a3, b3 = ops.adapters_linear_grad(g["dy"], g["x"], g["index"], g["A"], g["B"], g["scale"], base=g["dxb"],
                                          dtype=torch.float32)
    rest = torch.arange(100, device="cuda") != 4
    assert torch.equal(x3[rest], dx[rest]) and not x3[4].isfinite().any()
    assert torch.equal(a3[2], dA[2]) and not a3[1, 0].isfinite().any() and torch.equal(a3[1, 1:], dA[1, 1:])
    assert not b3[1].isfinite().any()


def test_repeats_and_streams(ops):
    """The same bits each time, on a stream of the caller's too."""
    c = make(1300, 6, 264, 264, 24, "bf16", "random")
    g, y = forward(ops, c)
    _, first = backward(ops, c)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y2 = ops.adapters_linear(g["base"], g["x"], g["index"], g["A"], g["B"], g["scale"])
        again = ops.adapters_linear_grad(g["dy"], g["x"], g["index"], g["A"], g["B"], g["scale"], base=g["dxb"],
                                         dtype=torch.float32)
    st.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("M", [7, 1200])
def test_graphs(ops, M):
    """Two captured graphs, replayed in turn on changing inputs, with eager calls between."""
    c = make(M, 4, 72, 136, 20, "fp16")
    g = dev(c)

    def step():
        y = ops.adapters_linear(g["base"], g["x"], g["index"], g["A"], g["B"], g["scale"])
        return (y, *ops.adapters_linear_grad(g["dy"], g["x"], g["index"], g["A"], g["B"], g["scale"], base=g["dxb"],
                                             dtype=torch.float32))

    step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for k in range(4):
        n = dev(make(M, 4, 72, 136, 20, "fp16", seed=k + 1))
        for name in g:
            g[name].copy_(n[name])
        want = step()
        graphs[k % 2].replay()
        graphs[1 - k % 2].replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(want, o))


def test_beside_the_integer_layer(ops):
    """A served batch: the merged integer layer's bf16 outputs, adapters of several requests added
    in place, row by row what each request's own weight gives within both roundings."""
    from integer_rank_adaptation_amd import synth

    d, n, r, M = 320, 320, 4, 40
    g = torch.Generator().manual_seed(5)
    W = torch.randn(d, n, generator=g).cuda() * 0.02
    A0, B0 = torch.randn(d, r, generator=g).cuda() * 0.02, torch.randn(r, n, generator=g).cuda() * 0.02
    st = ops.setup_layer(W, 8, synth.PHILOX_SEED, 7, synth.ALPHA)
    m = ops.merge_mul(st, A0, B0, 8, 8, synth.PHILOX_SEED, 7)
    c = make(M, 3, d, n, 16, "bf16", "random")
    xq, sx, rs = ops.quant_act(c["x"].float().cuda())
    Y, _ = ops.linear(xq, sx, rs, 16, m["m"], m["sbar"], d, split=m["split"])
    y = Y.view(torch.bfloat16)
    c["base"] = y.cpu()
    k = dev(c)
    out = ops.adapters_linear(y, k["x"], k["index"], k["A"], k["B"], k["scale"], out=y)
    want, spread = ref.forward(f64(c["base"]), f64(c["x"]), c["index"].numpy(), f64(c["A"]), f64(c["B"]), f64(c["scale"]))
    check(out, want, spread, "y")


@pytest.mark.parametrize("M,L,d,n,r", [(1100, 2, 16, 1 << 20, 3), (2200, 3, 1 << 19, 8, 5)])
def test_past_31_bits(ops, M, L, d, n, r):
    """Tensors of more than 2^31 bytes: rows go in several chunks.  Reference in fp64 on the device,
    a slice of columns at a time."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)
    x, A, B, base, dy = rand(M, n), rand(L, d, r), rand(L, r, n, std=n ** -0.5), rand(M, d), rand(M, d)
    ids = torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    s = torch.rand(L, generator=g, device="cuda") + 0.5
    assert max(M * n, M * d) * 2 > 1 << 31
    y = ops.adapters_linear(base, x, ids, A, B, s)
    dx, dA, dB = ops.adapters_linear_grad(dy, x, ids, A, B, s, dtype=torch.float32)

    def cols(width):
        return [slice(i, i + (1 << 16)) for i in range(0, width, 1 << 16)]

    for a in range(-1, L):
        rows = torch.nonzero(ids == a).flatten()
        if a < 0:
            assert torch.equal(y[rows], base[rows]) and not dx[rows].any()
            continue
        h = sum(x[rows][:, c].double() @ B[a][:, c].double().T for c in cols(n)) * s[a].double()
        dh = sum(dy[rows][:, c].double() @ A[a][c].double() for c in cols(d)) * s[a].double()
        # binary32 sums over n (d) products of about unit size: 2^-23 of the sum of magnitudes, at most
        # n 2^-23 times the mean product; two roundings to bf16 outputs
        for got, want, left in ((y, lambda c: base[rows][:, c].double() + h @ A[a][c].double().T, d),
                                (dx, lambda c: dh @ B[a][:, c].double(), n)):
            for c in cols(left):
                w = want(c)
                scale = w.abs().amax(1, keepdim=True) + 1.0
                assert ((got[rows][:, c].double() - w).abs() <= 2.0 ** -8 * (w.abs() + 2.0 ** -3 * scale)).all()
        for got, want, width in ((dA[a], lambda c: dy[rows][:, c].double().T @ h, d),
                                 (dB[a].T, lambda c: x[rows][:, c].double().T @ dh, n)):
            for c in cols(width):
                w = want(c)
                assert ((got[c].double() - w).abs() <= 2.0 ** -12 * (w.abs().max() + 1.0)).all()


@pytest.mark.parametrize("L", [1, 61, 62, 63, 64, 65, 127, 128, 130, 700, 4096])
@pytest.mark.parametrize("kind", ["random", "runs"])
def test_many_adapters(ops, L, kind):
    """Numbers of adapters around what a wave looks at when it finds its rows."""
    c = make(2600, L, 32, 40, 3, "bf16", kind)
    forward(ops, c)
    if L in (1, 63, 64, 130, 4096):
        backward(ops, c)


def test_long_lists(ops):
    """More rows than a listing block takes at a time, one adapter with nearly all of them."""
    c = make(20000, 3, 24, 16, 4, "fp16", "random")
    c["index"][c["index"] == 1] = 0
    c["index"][::997] = 1
    forward(ops, c)
    backward(ops, c)
