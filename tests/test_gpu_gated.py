"""The gated feed-forward layer and the calls on saved codes on the GPU, against the plain
definitions in binary64."""
import numpy as np
import pytest
import torch

from oracle import gated as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def ops():
    from integer_rank_adaptation_amd import ops

    return ops


def f64(t):
    return t.double().cpu().numpy()


def check(got, want, spread, what):
    """Within half a step of the type around `want`, and the spread."""
    f = torch.finfo(got.dtype)
    tol = spread + f.eps / 2 * np.maximum(np.abs(want) + spread, f.tiny)
    g = f64(got)
    bad = ~(np.abs(g - want) <= tol) & ~(np.isnan(g) & np.isnan(want))
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}, worst "
                           f"{np.nanmax(np.abs(g - want) / tol):.3g}")


def rand(shape, dt, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dt)


def split(T, E, seed, empty=0.3):
    """Ascending offsets of T rows over E groups, some without a row."""
    g = np.random.default_rng(seed)
    w = g.random(E) * (g.random(E) > empty)
    if w.sum() == 0:
        w[E // 2] = 1
    return np.concatenate(([0], np.round(np.cumsum(w) / w.sum() * T))).astype(np.int64)


def forward(ops, T, f, n, x="bf16", act="silu", E=0, save=False, seed=0):
    dt = DT[x]
    X, W = rand((T, n), dt, seed + 1), rand((max(E, 1), 2 * f, n), dt, seed + 2, 2 * n ** -0.5)
    off = split(T, E, seed) if E else None
    o = torch.from_numpy(off).cuda() if E else None
    got = ops.gated_linear(X.cuda(), o, W.cuda(), act=act, save=save)
    h, gu, eh, eg = ref.forward(f64(X), f64(W), off, act)
    check(got[0] if save else got, h, eh, "h")
    if save:
        check(got[1], gu, eg, "gu")
    return X, W, o, got


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 64, 100, 128, 129, 200, 300, 513])
@pytest.mark.parametrize("x,act,save", [("bf16", "silu", False), ("fp16", "gelu", True)])
def test_rows(ops, T, x, act, save):
    forward(ops, T, 136, 264, x, act, save=save)


@pytest.mark.parametrize("f", [8, 16, 24, 32, 40, 56, 64, 72, 120, 128, 136, 264])
@pytest.mark.parametrize("T,n", [(3, 72), (40, 136), (300, 72)])
def test_columns(ops, f, T, n):
    forward(ops, T, f, n, "bf16", "gelu", save=True)
    forward(ops, T, f, n, "fp16", "silu")


@pytest.mark.parametrize("n", [8, 16, 56, 64, 72, 120, 128, 136, 256, 1000, 2056])
@pytest.mark.parametrize("T", [5, 30, 150])
def test_contractions(ops, n, T):
    forward(ops, T, 72, n, "bf16", "silu", save=True)


# every launch of the tiled kernel: 64 x 64 tiles with four and two sets of waves, 128 x 128 with two sets and
# with two blocks to a unit, large ones alone (135 to 256), and with a rest of either kind behind them
@pytest.mark.parametrize("T,f", [(400, 320), (1000, 512), (1000, 1160), (2000, 1200), (2300, 1912), (4096, 2048),
                                 (4400, 2048), (5400, 2072)])
@pytest.mark.parametrize("x,act,save,E", [("bf16", "silu", True, 0), ("fp16", "gelu", False, 3), ("bf16", "gelu", True, 5)])
def test_tiles(ops, T, f, x, act, save, E):
    forward(ops, T, f, 72, x, act, E=E, save=save)


@pytest.mark.parametrize("T,E", [(1, 2), (7, 5), (40, 64), (64, 64), (300, 100), (1000, 7), (2000, 130)])
@pytest.mark.parametrize("x,act", [("bf16", "gelu"), ("fp16", "silu")])
def test_groups(ops, T, E, x, act):
    forward(ops, T, 104, 136, x, act, E=E, save=True)


@pytest.mark.parametrize("T", [10, 200])
def test_rows_in_no_group(ops, T):
    """Rows before the first and behind the last group are left as they are; wild offsets are forced in order."""
    X, W = rand((T, 72), DT["bf16"], 1), rand((3, 80, 72), DT["bf16"], 2, 0.2)
    a, b = 3, T - 4
    o = torch.tensor([a, 5, 5, b], device="cuda")
    H, GU = torch.full((T, 40), 7.0, dtype=DT["bf16"], device="cuda"), torch.full((T, 80), 7.0, dtype=DT["bf16"], device="cuda")
    h, gu = ops.gated_linear(X.cuda(), o, W.cuda(), save=True, out=(H, GU))
    assert h is H and gu is GU
    for t in (H, GU):
        assert (t[:a] == 7).all() and (t[b:] == 7).all()
    want, wgu, eh, eg = ref.forward(f64(X), f64(W), [a, 5, 5, b], "silu")
    check(H[a:b], want[a:b], eh[a:b], "h")
    check(GU[a:b], wgu[a:b], eg[a:b], "gu")
    wild = torch.tensor([-5, 6, 2, 1 << 40], device="cuda")  # as 0, 6, 6, T
    y = ops.gated_linear(X.cuda(), wild, W.cuda())
    want, _, eh, _ = ref.forward(f64(X), f64(W), [0, 6, 6, T], "silu")
    check(y, want, eh, "h")


@pytest.mark.parametrize("T", [6, 300])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_gates(ops, T, act):
    """Gates far from zero on both sides: H keeps its relative precision."""
    dt = DT["bf16"]
    X, W = rand((T, 64), dt, 3), rand((1, 48, 64), dt, 4, 0.3)
    X[0] *= 12
    X[1] *= 40
    X[2] *= 1e-3
    h = ops.gated_linear(X.cuda(), None, W.cuda(), act=act)
    want, _, eh, _ = ref.forward(f64(X), f64(W), None, act)
    check(h, want, eh, "h")


@pytest.mark.parametrize("T", [20, 400])
def test_non_finite_rows(ops, T):
    X, W = rand((T, 136), DT["bf16"], 5), rand((1, 128, 136), DT["bf16"], 6, 0.1)
    clean, cgu = ops.gated_linear(X.cuda(), None, W.cuda(), save=True)
    X[3, 130] = float("nan")
    X[7, 0] = float("inf")
    W[0, 64 + 5, 9] = float("nan")  # the up projection of column 5
    h, gu = ops.gated_linear(X.cuda(), None, W.cuda(), save=True)
    rows, cols = torch.ones(T, dtype=torch.bool), torch.ones(64, dtype=torch.bool)
    rows[[3, 7]] = False
    cols[5] = False
    assert h[3].isnan().all() and gu[3].isnan().all() and not gu[7].isfinite().any()
    assert torch.equal(h[rows.cuda()][:, cols.cuda()], clean[rows.cuda()][:, cols.cuda()]) and h[:, 5].isnan().all()
    assert torch.equal(gu[rows.cuda()][:, :64], cgu[rows.cuda()][:, :64])


def quantized(ops, v):
    q, s = ops.fp8_quant_act(v.cuda())
    return (q, s), ref.restore(q.view(torch.uint8).cpu().numpy(), s.cpu().numpy())


@pytest.mark.parametrize("T,f", [(1, 8), (3, 40), (17, 72), (100, 128), (33, 136), (64, 1000), (5, 5000)])
@pytest.mark.parametrize("x", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward(ops, T, f, x, act):
    dt = DT[x]
    dh, gu = rand((T, f), dt, 1, 0.3), rand((T, 2 * f), dt, 2, 2.5)
    dgu, h = ops.gated_linear_dgu(dh.cuda(), gu.cuda(), act=act)
    w, wh, tol, th = ref.backward(f64(dh), f64(gu), act)
    check(dgu, w, tol, "dgu")
    check(h, wh, th, "h")
    alone, none = ops.gated_linear_dgu(dh.cuda(), gu.cuda(), act=act, save=False)
    assert none is None and torch.equal(alone, dgu)
    pair, v = quantized(ops, gu.float())
    dgu, h = ops.gated_linear_dgu(dh.cuda(), pair, act=act)
    w, wh, tol, th = ref.backward(f64(dh), v, act)
    check(dgu, w, tol, "dgu of codes")
    check(h, wh, th, "h of codes")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_over_gates(ops, act):
    """All bf16 gates of magnitude up to 200, and infinities and NaN as the formulas give them."""
    bits = torch.arange(0, 0x4348, dtype=torch.int32).to(torch.int16)
    g = torch.cat((bits, bits + (-0x8000))).view(torch.bfloat16)
    g = g[: g.numel() // 8 * 8].reshape(-1, 8)
    dh, gu = torch.ones(g.shape, dtype=torch.bfloat16), torch.cat((g, torch.ones_like(g)), 1)
    dgu, h = ops.gated_linear_dgu(dh.cuda(), gu.cuda(), act=act)
    w, wh, tol, th = ref.backward(f64(dh), f64(gu), act)
    check(dgu, w, tol, "dgu")
    check(h, wh, th, "h")
    odd = torch.tensor([[float("inf"), float("nan"), 1.0, 0.0, -0.0, 3e38, -3e38, 1e-40]], dtype=torch.bfloat16)
    dgu, h = ops.gated_linear_dgu(torch.ones_like(odd).cuda(), torch.cat((odd, torch.ones_like(odd)), 1).cuda(), act=act)
    assert h[0, 0] == float("inf") and h[0, 1].isnan() and h[0, 3] == 0 and h[0, 5] > 2e38 and h[0, 6] == 0
    assert dgu[0, 8] == float("inf") and dgu[0, 1].isnan() and dgu[0, 3] == 0.5 and dgu[0, 2].isfinite()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_restore_every_code(ops, dt):
    """Every code under scales over the whole range, and of other row lengths."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(14, 1)
    scale = torch.full((14, 4), 127, dtype=torch.uint8)
    scale[:, 0] = torch.tensor([0, 1, 2, 60, 100, 112, 120, 127, 134, 135, 140, 246, 254, 255], dtype=torch.uint8)
    scale[:, 1] = scale[:, 0].flip(0)
    v = ref.restore(codes.numpy(), scale.numpy())
    got = ops.fp8_dequant_act(codes.view(torch.float8_e4m3fn).cuda(), scale.cuda(), dt).cpu()
    with np.errstate(over="ignore"):
        # binary32 first (exact but for its own range), then the type, fp16 up to its largest number
        w = torch.from_numpy(v).float()
    if dt == torch.float16:
        w = torch.where(w.isnan(), w, w.clamp(-65504, 65504))
    want = w.to(dt)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(got, 0, 1, -1), torch.nan_to_num(want, 0, 1, -1))


@pytest.mark.parametrize("T,n", [(1, 16), (3, 48), (7, 128), (5, 144), (100, 640), (33, 1424), (2, 5008)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
def test_restore(ops, T, n, dt):
    pair, v = quantized(ops, rand((T, n), dt, 1, 3.0))
    out = torch.empty((T, n), dtype=dt, device="cuda")
    assert ops.fp8_dequant_act(*pair, dt, out=out) is out
    assert np.array_equal(f64(out), v)  # exact: the type holds them


@pytest.mark.parametrize("T,d,n,E", [
    (1, 8, 16, 0), (5, 16, 48, 0), (64, 72, 144, 0), (65, 136, 128, 0), (300, 72, 640, 0), (1000, 264, 400, 0),
    (100, 72, 144, 7), (333, 136, 272, 20), (700, 1000, 1424, 5), (2000, 640, 640, 3), (129, 2304, 4000, 0),
])
@pytest.mark.parametrize("x", ["bf16", "fp16"])
def test_dw(ops, T, d, n, E, x):
    dt = DT[x]
    dy = rand((T, d), dt, 1, 0.2)
    X = rand((T, n), dt, 2)
    X[:, 3] *= 30
    pair, v = quantized(ops, X)
    off = split(T, E, 4) if E else None
    o = torch.from_numpy(off).cuda() if E else None
    want, tol = ref.dw(f64(dy), v, off)
    for kind in (dt, torch.float32):
        got = ops.grouped_linear_dw(dy.cuda(), pair, o, dtype=kind)
        assert got.dtype == kind
        check(got, want, tol, f"dw {kind}")


def test_dw_edges(ops):
    """Blocks of tiny and of huge numbers in one row, a block with a NaN, codes past fp16's range, no rows."""
    dt = torch.bfloat16
    dy, X = rand((70, 16), dt, 1), rand((70, 400), dt, 2)
    X[:, :128] *= 1e-30
    X[:, 128:256] *= 1e25
    pair, v = quantized(ops, X)
    want, tol = ref.dw(f64(dy), v, None)
    check(ops.grouped_linear_dw(dy.cuda(), pair, None, dtype=torch.float32), want, tol, "range")
    X[7, 300] = float("nan")
    pair, _ = quantized(ops, X)
    got = ops.grouped_linear_dw(dy.cuda(), pair, None, dtype=torch.float32).cpu()
    assert got[0, :, 256:384].isnan().all() and got[0, :, :256].isfinite().all() and got[0, :, 384:].isfinite().all()
    half = torch.zeros(3, 128, dtype=torch.float16)
    half[1, 5], half[2, 6] = 65504, -65504
    pair, _ = quantized(ops, half)
    got = ops.grouped_linear_dw(torch.eye(3, 8, dtype=torch.float16).cuda(), pair, None).cpu()
    assert got[0, 1, 5] == 65504 and got[0, 2, 6] == -65504 and got.abs().sum(dtype=torch.float64) == 2 * 65504
    q, s = torch.empty(0, 32, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(0, 4, dtype=torch.uint8, device="cuda")
    got = ops.grouped_linear_dw(torch.empty(0, 8, dtype=dt, device="cuda"), (q, s), torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert got.shape == (2, 8, 32) and not got.any()


def test_streams(ops):
    X, W, _, (h, gu) = forward(ops, 300, 136, 264, "bf16", "silu", save=True)
    dh = rand((300, 136), DT["bf16"], 9).cuda()
    x, w = X.cuda(), W.cuda()
    dgu, _ = ops.gated_linear_dgu(dh, gu)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        h2, gu2 = ops.gated_linear(x, None, w, save=True)
        dgu2, _ = ops.gated_linear_dgu(dh, gu2)
    st.synchronize()
    assert torch.equal(h, h2) and torch.equal(gu, gu2) and torch.equal(dgu, dgu2)


@pytest.mark.parametrize("T,E", [(24, 3), (600, 3), (4400, 0)])
def test_training_step(ops, T, E):
    """An adapted gated feed-forward layer trained on saved codes: forward, every gradient, in one go,
    captured in a graph and replayed on changing inputs; each part against its definition on the
    very tensors it was given."""
    from oracle import adapters as lora

    dt, f, n, r = torch.bfloat16, 208, 144, 12
    g = E or 1

    def inputs(seed):
        return dict(x=rand((T, n), dt, seed), w=rand((g, 2 * f, n), dt, 50, n ** -0.5), wd=rand((g, n, f), dt, 51, f ** -0.5),
                    dy=rand((T, n), dt, seed + 1, 0.1), A=rand((3, n, r), dt, 52, 0.1), B=rand((3, r, f), dt, 53, f ** -0.5),
                    s=torch.tensor([0.5, 1.0, 2.0]), ids=torch.arange(T, dtype=torch.int32) % 4 - 1)

    off = split(T, E, 3) if E else None
    o = torch.from_numpy(off).cuda() if E else None
    c = {k: v.cuda() for k, v in inputs(0).items()}

    def step():
        h, gu = ops.gated_linear(c["x"], o, c["w"], save=True)
        y = ops.adapters_linear(ops.grouped_linear(h, o, c["wd"]), h, c["ids"], c["A"], c["B"], c["s"])
        sx, sgu = ops.fp8_quant_act(c["x"]), ops.fp8_quant_act(gu)  # all that the backward keeps
        dh = ops.grouped_linear_dx(c["dy"], o, c["wd"])
        dgu, h2 = ops.gated_linear_dgu(dh, sgu)
        dh2, dA, dB = ops.adapters_linear_grad(c["dy"], h2, c["ids"], c["A"], c["B"], c["s"], base=dh,
                                               dtype=torch.float32)
        dgu2, _ = ops.gated_linear_dgu(dh2, sgu, save=False)
        dwd = ops.grouped_linear_dw(c["dy"], h2, o)
        return dict(h=h, gu=gu, y=y, dgu=dgu, h2=h2, dh=dh, dh2=dh2, dA=dA, dB=dB, dgu2=dgu2, dwd=dwd,
                    dx=ops.grouped_linear_dx(dgu2, o, c["w"]), dw=ops.grouped_linear_dw(dgu2, sx, o, dtype=torch.float32))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (10, 20, 30):
        for k, v in inputs(seed).items():
            c[k].copy_(v)
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(out[k], want[k]), k
    cpu = {k: v.cpu() for k, v in c.items()}
    h, gu, eh, eg = ref.forward(f64(cpu["x"]), f64(cpu["w"]), off, "silu")
    check(out["h"], h, eh, "h")
    check(out["gu"], gu, eg, "gu")
    _, v = quantized(ops, out["gu"])
    w, wh, tol, th = ref.backward(f64(out["dh2"]), v, "silu")
    check(out["dgu2"], w, tol, "dgu")
    check(out["h2"], wh, th, "h again")
    _, v = quantized(ops, cpu["x"])
    w, tol = ref.dw(f64(out["dgu2"]), v, off)
    check(out["dw"], w, tol, "dw")
    w, tol = lora.backward(f64(out["dh"]), f64(cpu["dy"]), f64(out["h2"]), cpu["ids"].numpy(), f64(cpu["A"]), f64(cpu["B"]),
                           f64(cpu["s"]))
    for k, t in (("dx", "dh2"), ("dA", "dA"), ("dB", "dB")):
        check(out[t], w[k], tol[k], t)


def test_outputs_past_31_bits(ops):
    """Projections, gradients and restored codes of more than 2^31 bytes: the first, some middle and the
    last rows, at the first and last columns."""
    T, f, n = 41003, 13120, 32
    assert 2 * T * 2 * f > 1 << 31
    X, W = rand((T, n), DT["bf16"], 1).cuda(), rand((1, 2 * f, n), DT["bf16"], 2, 2 * n ** -0.5).cuda()
    h, gu = ops.gated_linear(X, None, W, save=True)
    dh = torch.randn(T, f, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(torch.bfloat16)
    dgu, h2 = ops.gated_linear_dgu(dh, gu)
    pair = ops.fp8_quant_act(gu)
    dguq, _ = ops.gated_linear_dgu(dh, pair)
    back = ops.fp8_dequant_act(*pair, torch.bfloat16)
    rows = torch.tensor([0, 1, 127, 128, 20000, 20479, 20480, T - 4, T - 3, T - 2, T - 1], device="cuda")
    for a in (0, f // 2 - 80, f - 128):
        c = torch.cat((torch.arange(a, a + 128), torch.arange(f + a, f + a + 128))).cuda()
        at = lambda t, k=c: t[rows][:, k]
        want, wgu, eh, eg = ref.forward(f64(X[rows]), f64(W[:, c]), None, "silu")
        check(at(h, c[:128]), want, eh, "h")
        check(at(gu), wgu, eg, "gu")
        w, wh, tol, th = ref.backward(f64(at(dh, c[:128])), f64(at(gu)), "silu")
        check(at(dgu), w, tol, "dgu")
        check(at(h2, c[:128]), wh, th, "h again")
        assert (at(back).double() - at(gu).double()).abs().max() <= 2.0 ** -4 * at(gu).double().abs().max()
        w, _, tol, _ = ref.backward(f64(at(dh, c[:128])), f64(at(back)), "silu")
        check(at(dguq), w, tol, "dgu of codes")


@pytest.mark.parametrize("T", [3, 300])
def test_weights_past_31_bits(ops, T):
    f, n = (1 << 19) - 8, 1032
    X = rand((T, n), DT["bf16"], 1).cuda()
    W = torch.randn(1, 2 * f, n, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda",
                    dtype=torch.bfloat16) * n ** -0.5
    assert 2 * W.numel() > 1 << 31
    h, gu = ops.gated_linear(X, None, W, act="gelu", save=True)
    for a in (0, f // 2, f - 136):
        c = torch.cat((torch.arange(a, a + 136), torch.arange(f + a, f + a + 136))).cuda()
        want, wgu, eh, eg = ref.forward(f64(X), f64(W[:, c]), None, "gelu")
        check(h[:, c[:136]], want, eh, "h")
        check(gu[:, c], wgu, eg, "gu")


def test_two_threads(ops):
    """Calls of two threads at once, each on a stream of its own."""
    import threading

    X, W = rand((200, 264), DT["fp16"], 1).cuda(), rand((1, 272, 264), DT["fp16"], 2, 264 ** -0.5).cuda()
    A, B = rand((3, 264, 20), DT["fp16"], 3, 0.1).cuda(), rand((3, 20, 136), DT["fp16"], 4, 0.1).cuda()
    ids, s = torch.arange(200, dtype=torch.int32).cuda() % 4 - 1, torch.ones(3).cuda()

    def work():
        h, gu = ops.gated_linear(X, None, W, save=True)
        y = ops.adapters_linear(X, h, ids, A, B, s)
        return [y, ops.gated_linear_dgu(h, ops.fp8_quant_act(gu))[0],
                *ops.adapters_linear_grad(y, h, ids, A, B, s, dtype=torch.float32)]

    want = work()
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def run(k):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(20):
                    got[k] = work()
            st.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
