"""On the GPU, through the extension module and through ctypes: tensors with a
forward-mode tangent are refused, and primals give what they gave."""
import pytest
import torch
from torch.autograd import forward_ad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("fast", [True, False])
def test_tangents_are_refused(fast, monkeypatch):
    from mixed_precision_weight_page_amd import pagedweight as pwb
    if not fast:
        monkeypatch.setattr(pwb, "_fast", None)
    x, w = torch.randn(4, 32, device="cuda").bfloat16(), torch.randn(2, 8, 32, device="cuda").bfloat16()
    n, off = torch.ones(32, device="cuda"), torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda")
    bias, tile = torch.randn(8, device="cuda"), pwb.quantize_fp8(w[0], "tile")
    place, g = torch.arange(4, dtype=torch.int32, device="cuda")[:, None], torch.ones(4, 1, device="cuda")
    calls = {"linear": lambda d: pwb.linear(d(x), w[0]), "norm": lambda d: pwb.rms_norm(d(x), n), "weight": lambda d: pwb.rms_norm(x, d(n)),
             "quantize": lambda d: pwb.quantize_fp8(d(x)), "bias": lambda d: pwb.linear_fp8(pwb.quantize_fp8(x), tile, bias=d(bias)),
             "grouped": lambda d: pwb.grouped_linear(d(x), off, w), "join": lambda d: pwb.join_routes(d(x), place, g)}
    want = {name: call(lambda t: t) for name, call in calls.items()}
    with forward_ad.dual_level():
        for name, call in calls.items():
            with pytest.raises(ValueError, match="tangent"):
                call(lambda t: forward_ad.make_dual(t, torch.ones_like(t)))
            got = call(lambda t: t)
            for a, b in zip(got, want[name]) if isinstance(got, tuple) else ((got, want[name]),):
                assert torch.equal(a.float(), b.float())
