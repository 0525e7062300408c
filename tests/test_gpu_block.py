"""GPU tests of the calls around the expert layer as a block uses them:
streams given by handle, captured and replayed blocks."""
import pytest
import torch

import synth
from layer_cases import log, make_layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


GATE = dict(score="sigmoid", n_group=4, topk_group=2, group_score="top2", renorm=True, scale=2.5)


class Block:
    """A layer of 16 experts with pages of every width, its router's and its
    shared expert's weights, and T tokens."""
    def __init__(self, T, seed=1, layout="eq2", **shape):
        wl = synth.WORKLOADS["decode_fine"].scaled(name="block", T=max(T, 1), **{**dict(E=16, d=256, F=384, k=4), **shape})
        self.wl = wl
        self.layer, _ = make_layer(wl, synth.expert_weights(wl), max_tokens=max(T, 1), layout=layout)
        self.bits = [(3, 4, 8)[e % 3] if layout == "eq2" else 1 + e % 8 for e in range(wl.E)]
        self.layer.quantize_experts(self.bits)
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
        self.gate_w = (rand(wl.E, wl.d) / 16).bfloat16().cuda()
        self.shared = ((rand(2 * 200, wl.d) / 16).bfloat16().cuda(), (rand(wl.d, 200) / 14).bfloat16().cuda())
        self.bias = (rand(wl.E) * 0.1).cuda()
        self.batches = [(rand(T, wl.d).bfloat16().cuda(), rand(T, wl.d).bfloat16().cuda()) for _ in range(3)]

    def __call__(self, x, residual, **kw):
        return self.layer.moe_block(x, self.gate_w, shared=self.shared, residual=residual, bias=self.bias, **{**GATE, **kw})


def test_stream_zero_is_the_default_stream(monkeypatch):
    """The handle 0 given while another stream is the current one."""
    from mixed_precision_weight_page_amd import linear
    from mixed_precision_weight_page_amd import pagedweight as pwb
    b = Block(24)
    x, res = b.batches[0]
    want = b(x, res)
    logits = linear(x, b.gate_w, out_dtype=torch.float32)
    torch.cuda.synchronize()
    used, raw = [], pwb._raw_stream
    monkeypatch.setattr(pwb, "_raw_stream", lambda dev: used.append(raw(dev)) or used[-1])
    with torch.cuda.stream(torch.cuda.Stream()):
        outs = [b(x, res, stream=0), linear(x, b.gate_w, out_dtype=torch.float32, stream=0),
                b.layer.route_gated(logits, bias=b.bias, stream=0, **GATE),
                b.layer.moe_forward_routed(x, want[1], want[2], stream=0)]
    torch.cuda.synchronize()
    assert used == [0] * 8   # five calls of the block, three others
    for got, w in zip(outs[0], want):
        assert torch.equal(got, w)
    assert torch.equal(outs[1], logits)
    for got, w in zip(outs[2], want[1:]):
        assert torch.equal(got, w)
    assert torch.equal(outs[3], b.layer.moe_forward_routed(x, want[1], want[2]))


def test_tensors_that_require_a_gradient():
    """Refused one by one where gradients are recorded; under no_grad the
    same tensors give the same block."""
    b = Block(6)
    x, res = b.batches[0]
    want = b(x, res)
    for t in (x, res, b.gate_w, b.bias, *b.shared):
        t.requires_grad_()
        with pytest.raises(ValueError, match="forward only"):
            b(x, res)
        t.requires_grad_(False)
    for t in (x, res, b.gate_w, b.bias, *b.shared):
        t.requires_grad_()
    with torch.no_grad():
        got = b(x, res)
    for g, w in zip(got, want):
        assert torch.equal(g, w) and not g.requires_grad
