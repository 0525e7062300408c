"""A call on a side stream refuses what the same call on the current stream
refuses, in the same words, and tells the allocator about every tensor it was
given. No call here touches a GPU."""
import contextlib

import pytest
import torch

from mixed_precision_weight_page_amd import pagedweight as pwb

E4M3 = torch.float8_e4m3fn


@pytest.fixture
def side(monkeypatch):
    """A stream that is not the current one; tensors pass as if they were on a GPU."""
    stream = object()
    monkeypatch.setattr(pwb, "_other_stream", lambda s: s)
    monkeypatch.setattr(pwb, "_here", lambda t, name: (0, None))
    monkeypatch.setattr(pwb, "_on_gpu", lambda t, dev, name: None)
    monkeypatch.setattr(pwb, "_fast", None)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return stream


def refusals():
    x = torch.zeros(2, 32).bfloat16()
    pair = (torch.zeros(2, 32).to(E4M3), torch.zeros(2, 1))
    tile = (torch.zeros(8, 32).to(E4M3), torch.zeros(1, 1))
    off = torch.zeros(4, dtype=torch.int32)
    return {
        "norm of a row": lambda s: pwb.rms_norm(x[0], stream=s),
        "norm of nothing": lambda s: pwb.rms_norm(None, stream=s),
        "norm, out a tensor": lambda s: pwb.rms_norm(x, out=x, out_dtype=E4M3, stream=s),
        "norm, out a pair": lambda s: pwb.rms_norm(x, out=pair, out_dtype=torch.float32, stream=s),
        "quantize, out a tensor": lambda s: pwb.quantize_fp8(x, out=pair[0], stream=s),
        "quantize, out one element": lambda s: pwb.quantize_fp8(x[:1, :1], out=pair[0][:1, :1], stream=s),
        "quantize, out three": lambda s: pwb.quantize_fp8(x, out=(*pair, x), stream=s),
        "quantize, block": lambda s: pwb.quantize_fp8(x, "column", stream=s),
        "linear_fp8, x a tensor": lambda s: pwb.linear_fp8(x, tile, stream=s),
        "linear_fp8, x nothing": lambda s: pwb.linear_fp8(None, tile, stream=s),
        "linear_fp8, w a tensor": lambda s: pwb.linear_fp8(pair, x, stream=s),
        "linear_fp8, act": lambda s: pwb.linear_fp8(pair, tile, act="tanh", stream=s),
        "linear_fp8, y": lambda s: pwb.linear_fp8(pair, tile, y=x, stream=s),
        "grouped, w a pair": lambda s: pwb.grouped_linear(x, off, tile, stream=s),
        "grouped, w nothing": lambda s: pwb.grouped_linear(x, off, None, stream=s),
        "grouped, offsets": lambda s: pwb.grouped_linear(x, None, x[None], stream=s),
        "routes": lambda s: pwb.group_routes(off, 3, stream=s),
        "routes of nothing": lambda s: pwb.group_routes(None, 3, stream=s),
        "join": lambda s: pwb.join_routes(x, off, off, stream=s),
        "experts, both kinds": lambda s: pwb.moe_experts(x, off[None], off, x[None], tile, stream=s),
        "experts, no weights": lambda s: pwb.moe_experts(x, off[None], off, None, None, stream=s),
        "experts, no ids": lambda s: pwb.moe_experts(x, None, off, x[None], x[None], stream=s),
    }


@pytest.mark.parametrize("name", list(refusals()))
def test_the_same_refusals(side, name):
    call = refusals()[name]
    with pytest.raises(ValueError) as here:
        call(None)
    with pytest.raises(ValueError) as there:
        call(side)
    assert str(there.value) == str(here.value) and "ambiguous" not in str(here.value)


def test_every_tensor_is_recorded(side, monkeypatch):
    seen = []
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append((t, s)), raising=False)
    t = [torch.zeros(1) for _ in range(6)]
    assert pwb._call_on(side, (t[0], None, (t[1], t[2]), pwb.Fp8(t[3], t[4]), [(t[5], None)], "none", 3), lambda: 7) == 7
    assert len(seen) == 6 and all(a is b and s is side for (a, s), b in zip(seen, t))


def test_a_call_that_raises_midway_has_them_recorded_too(side, monkeypatch):
    """Part of it may be running on the stream already."""
    seen = []
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True), raising=False)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append(t), raising=False)
    t = torch.zeros(1)

    def call():
        raise ValueError("midway")

    with pytest.raises(ValueError, match="midway"):
        pwb._call_on(side, (t,), call)
    assert len(seen) == 1 and seen[0] is t
