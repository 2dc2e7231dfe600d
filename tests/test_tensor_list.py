"""Lists of gradients are read in one compiled pass (CPU: the host tensors' device is -1; GPU: the
calls on top of it)."""
import ctypes
import weakref

import pytest
import torch

from integer_rank_adaptation_amd import binding as B
from integer_rank_adaptation_amd import ops

CODES = {torch.bfloat16: B.INTLORA_BF16, torch.float16: B.INTLORA_FP16, torch.float32: B.INTLORA_FP32}


class Counted(torch.Tensor):
    """Counts the Python calls that touch a tensor."""

    calls = 0

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        Counted.calls += 1
        return super().__torch_function__(func, types, args, kwargs or {})


def _some():
    return [torch.arange(6.0).view(2, 3), torch.zeros(0, 5), torch.zeros(7, dtype=torch.bfloat16)[2:],
            torch.nn.Parameter(torch.ones(3, 1, 4).half()), torch.tensor(2.0), torch.zeros(1 << 20)]


def test_addresses_sizes_and_types():
    ts = _some()
    ptrs, numel, types = ops._read("grads", ts, -1)
    assert list(numel) == [t.numel() for t in ts] and list(types) == [CODES[t.dtype] for t in ts]
    assert [p or 0 for p in ptrs] == [t.data_ptr() for t in ts]
    assert isinstance(ptrs, ctypes.Array) and ops._tensors("grads", iter(ts)) == ts
    assert [len(a) for a in ops._read("grads", [], -1)] == [0, 0, 0]


def test_no_python_call_per_tensor():
    ts = [t.detach().as_subclass(Counted) for t in _some()]
    Counted.calls = 0
    ops._read("grads", ts, -1)
    assert Counted.calls == 0


@pytest.mark.parametrize("bad,error,text", [
    (torch.zeros(4, 4).t(), ValueError, "contiguous tensors on the current device"),
    (torch.zeros(4, 4)[:, :2], ValueError, "contiguous tensors on the current device"),
    (torch.zeros(3, dtype=torch.float64), ValueError, "expected bf16, fp16 or fp32 tensors, got torch.float64"),
    (torch.zeros(3, dtype=torch.int16), ValueError, "got torch.int16"),
    (torch.eye(3).to_sparse(), (ValueError, RuntimeError), None),
    (None, TypeError, "expected tensors, got NoneType"),
    (3.0, TypeError, "expected tensors, got float"),
])
def test_refusals(bad, error, text):
    for ts in ([bad], [torch.zeros(2), bad], [bad, torch.zeros(2)]):
        with pytest.raises(error, match=text):
            ops._read("grads", ts, -1)
    with pytest.raises(ValueError, match="grads: expected a list"):
        ops._tensors("grads", torch.zeros(2, 2))
    for t in (torch.zeros(2), torch.zeros(2, device="meta")):  # on no GPU
        with pytest.raises(ValueError, match="out: expected contiguous tensors on the current device"):
            ops._read("out", [t], 0)


def test_tensors_of_an_iterator_live_until_the_call_is_enqueued(monkeypatch):
    """Tensors that only the iterator made: their memory may not go back (and become the
    workspace) before the kernels that read them are enqueued."""
    made, seen = [], []

    def temporaries():
        for i in range(3):
            t = torch.ones(4 + i)
            made.append(weakref.ref(t))
            yield t

    def sumsq(ptrs, numel, types, dev):
        seen.append([r() is not None for r in made])
        return torch.zeros(1, dtype=torch.float64)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(ops, "_sumsq", sumsq)
    ops.grad_sumsq(temporaries())
    monkeypatch.setattr(ops, "_clip", lambda *a: seen.append([r() is not None for r in made]))
    ops.clip_grad_norm(temporaries(), 1.0)
    assert seen == [[True] * 3, [False] * 3 + [True] * 3, [False] * 3 + [True] * 3]


@pytest.mark.gpu
def test_temporary_gradients_and_outputs():
    gs = [torch.full((1 << 16,), float(i + 1), device="cuda") for i in range(8)]
    total = (1 << 16) * sum((2.0 * (i + 1)) ** 2 for i in range(8))
    out = [torch.zeros_like(g) for g in gs]
    for _ in range(3):
        norm = ops.clip_grad_norm((2 * g for g in gs), 1.0, out=(o.view(-1) for o in out))
        s = ops.grad_sumsq(2 * g for g in gs)
        assert float(s) == total and abs(float(norm) - total**0.5) <= total**0.5 * 2.0**-23
        for i, o in enumerate(out):
            want = 2.0 * (i + 1) / (total**0.5 + 1e-6)  # the factor and the product are rounded to binary32
            assert (o.double() - want).abs().max() <= want * 2.0**-23 * 1.001


@pytest.mark.gpu
def test_calls_make_no_python_call_per_tensor():
    gs = [torch.full((5 + i % 7,), 0.5, device="cuda", dtype=(torch.float16, torch.float32)[i % 2]).as_subclass(Counted)
          for i in range(300)]
    out = [torch.zeros_like(g) for g in gs]
    n = sum(g.numel() for g in gs)
    Counted.calls = 0
    norm = ops.clip_grad_norm(gs, 1.0, out=out)
    total = ops.grad_sumsq(gs)
    ops.grad_clip(gs, total, 1.0)
    assert Counted.calls == 0
    assert abs(float(norm) - 0.5 * n**0.5) <= 2.0**-24 * n**0.5 and float(total) == 0.25 * n
    c = 1.0 / (0.5 * n**0.5 + 1e-6)
    for g, o in zip(gs, out):
        assert torch.equal(g, o) and abs(float(o[0]) - 0.5 * c) <= 0.5 * c * torch.finfo(o.dtype).eps


@pytest.mark.gpu
def test_outputs_of_other_sizes_and_types_are_refused():
    g = [torch.zeros(4, device="cuda"), torch.zeros(6, device="cuda", dtype=torch.float16)]
    for out in ([g[0]], [torch.zeros(4, device="cuda"), torch.zeros(7, device="cuda", dtype=torch.float16)],
                [torch.zeros(4, device="cuda"), torch.zeros(6, device="cuda", dtype=torch.bfloat16)],
                [torch.zeros(4, device="cuda"), torch.zeros(6, dtype=torch.float16)], []):
        with pytest.raises(ValueError, match="out: expected"):
            ops.clip_grad_norm(g, 1.0, out=out)
