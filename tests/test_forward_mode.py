"""Tensors with a forward-mode tangent are refused: the calls have no
derivative, and would return a result without it. Host only."""
import pytest
import torch
from torch.autograd import forward_ad

from mixed_precision_weight_page_amd import pagedweight as pwb

E4M3 = torch.float8_e4m3fn


def calls(mark):
    """The calls, with mark(t) as the one tensor that may carry a tangent."""
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    b = lambda *s: f(*s).bfloat16()  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pair, tile = lambda s: (f(2, 32).to(E4M3), s), (f(8, 32).to(E4M3), f(1, 1))
    return {
        "linear x": lambda: pwb.linear(mark(b(2, 16)), b(8, 16)),
        "norm x": lambda: pwb.rms_norm(mark(b(2, 32))),
        "norm weight": lambda: pwb.rms_norm(b(2, 32), mark(f(32))),
        "norm residual": lambda: pwb.rms_norm(b(2, 32), residual=mark(f(2, 32))),
        "quantize x": lambda: pwb.quantize_fp8(mark(f(2, 32))),
        "linear_fp8 scales": lambda: pwb.linear_fp8(pair(mark(f(2, 1))), tile),
        "linear_fp8 bias": lambda: pwb.linear_fp8(pair(f(2, 1)), tile, bias=mark(f(8))),
        "grouped x": lambda: pwb.grouped_linear(mark(b(2, 32)), i(2), b(1, 8, 32)),
        "grouped w": lambda: pwb.grouped_linear(b(2, 32), i(2), mark(b(1, 8, 32))),
        "join g": lambda: pwb.join_routes(b(2, 32), i(2, 1), mark(f(2, 1))),
    }


@pytest.fixture
def as_on_gpu(monkeypatch):
    monkeypatch.setattr(pwb, "_here", lambda t, name: (0, None))
    monkeypatch.setattr(pwb, "_fast", None)
    on_gpu = pwb._on_gpu

    def passes(t, dev, name):   # all but that the tensors are on the CPU
        try:
            on_gpu(t, dev, name)
        except ValueError as e:
            if "CUDA" not in str(e):
                raise
    monkeypatch.setattr(pwb, "_on_gpu", passes)


class Passed(Exception):
    pass


@pytest.mark.parametrize("name", list(calls(None)))
def test_tangents_are_refused(as_on_gpu, monkeypatch, name):
    def no_call():
        raise Passed
    monkeypatch.setattr(pwb, "lib", no_call)
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            calls(lambda t: forward_ad.make_dual(t, torch.ones_like(t)))[name]()
        with torch.no_grad(), pytest.raises(ValueError, match="tangent"):   # which does not switch these off
            calls(lambda t: forward_ad.make_dual(t, torch.ones_like(t)))[name]()
        # without one, and with one taken off, on to the library
        for mark in (lambda t: t, lambda t: forward_ad.unpack_dual(forward_ad.make_dual(t, torch.ones_like(t))).primal):
            with pytest.raises(Passed):
                calls(mark)[name]()
    with pytest.raises(Passed):
        calls(lambda t: t)[name]()
