"""CPU: what the binding hands to the library under dropout and for 8-bit
linears.  The library and the device are replaced by a recorder, and CPU
tensors pass for GPU ones, so that a buffer which no kernel may be given is
seen to be refused (or passed on) without a GPU."""

import dataclasses

import pytest
import torch

from bit_quantized_finetuning_nf4_amd import ops

M, N, K, R = 4, 64, 128, 8
DROP = ops.Dropout(0.1, 1)


class Gpu(torch.Tensor):
    is_cuda = True


def t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(Gpu)


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Recorder:
        def __getattr__(self, name):
            if name == "qlora_workspace_bytes":
                return lambda *a: 256
            return lambda *a: seen.append(name) or 0
    monkeypatch.setattr(ops, "lib", lambda: Recorder())
    monkeypatch.setattr(ops, "_on_current", lambda device: None)
    monkeypatch.setattr(ops, "_stream", lambda: 0)
    return seen


def nf4():
    return ops.QuantizedWeight(N, K, t(N * K // 2, torch.uint8), t(N * K // 64, torch.uint8), t(1, torch.float32))


def i8():
    return ops.Int8Weight(N, K, t((N, 128), torch.int8), t(N, torch.float32))


def forward(kind, w=None, **kw):
    f, w = (ops.linear_fwd, w or nf4()) if kind == "nf4" else (ops.i8_linear_fwd, w or i8())
    return f(w, t((M, K)), t((R, K)), t((N, R)), 16.0, save_u=True, drop=DROP, **kw)


def backward(kind, w=None, **kw):
    f, w = (ops.linear_bwd, w or nf4()) if kind == "nf4" else (ops.i8_linear_bwd, w or i8())
    return f(w, t((M, K)), t((M, N)), t((R, K)), t((N, R)), 16.0, drop=DROP, **kw)


def bad(shape, dtype):
    """Short, of the wrong type, strided."""
    rows, cols = shape
    return {"short": t((rows, cols - 8), dtype), "one row less": t((rows - 1, cols), dtype),
            "flat": t(rows * cols, dtype), "type": t(shape, torch.float16),
            "strided": t((cols, rows), dtype).t(), "cpu": torch.zeros(shape, dtype=dtype)}


@pytest.mark.parametrize("kind", ["nf4", "i8"])
@pytest.mark.parametrize("fault", ["short", "one row less", "flat", "type", "strided", "cpu"])
def test_outputs(calls, kind, fault):
    good = dict(out=t((M, N)), u_out=t((M, R)), ws=t(1024, torch.uint8))
    assert [x.data_ptr() for x in forward(kind, **good)] == [good["out"].data_ptr(), good["u_out"].data_ptr()]
    assert len(calls) == 1
    for name, shape in (("out", (M, N)), ("u_out", (M, R))):
        with pytest.raises(ValueError):
            forward(kind, **{**good, name: bad(shape, torch.bfloat16)[fault]})
    good = dict(dX=t((M, K)), dA=t((R, K), torch.float32), dB=t((N, R), torch.float32), U=t((M, R)))
    backward(kind, **good)
    assert len(calls) == 2
    for name, x in good.items():
        with pytest.raises(ValueError):
            backward(kind, **{**good, name: bad(tuple(x.shape), x.dtype)[fault]})
    assert len(calls) == 2   # nothing refused was launched


@pytest.mark.parametrize("call", [forward, backward])
def test_weights(calls, call):
    q = nf4()
    for change in (dict(codes=q.codes[:-1]), dict(absmax_q=q.absmax_q[:-1]), dict(group_scale=q.group_scale[:0]),
                   dict(codes=q.codes.to(torch.int8)), dict(absmax_q=q.absmax_q.int()),
                   dict(group_scale=q.group_scale.double()), dict(absmax_q=torch.zeros(N * K // 64, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call("nf4", dataclasses.replace(q, **change))
    w = i8()
    for change in (dict(codes=w.codes[:-1]), dict(scale=w.scale[:-1]), dict(scale=w.scale.double())):
        with pytest.raises(ValueError):
            call("i8", dataclasses.replace(w, **change))
    assert not calls
    # a larger buffer (a slice of a pool, say) holds the weight too
    call("nf4", dataclasses.replace(q, codes=t(N * K, torch.uint8)))
    assert len(calls) == 1
