"""GPU tests of pw_moe_forward_routed (the experts' products for given ids
and weights) and of the whole block (PagedMoELayer.moe_block), against
float64 products of the dequantized weights. fp32 outputs: the layer's
tolerance; bf16 outputs: that and the rounding, half a step of 2^-7 of each
element (2^-8 in the norm as well)."""
import pytest
import torch

import synth
from layer_cases import YTOL_MAX, YTOL_NORM, cpu_threads, log, make_layer
from oracle import bitplane, quant

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cpu_threads()


def weights64(masters, bits, layout):
    """The dequantized (w1, w3, w2) of every expert in float64."""
    if layout == "bitplane":
        get = bitplane.experts(*masters, bits)
        return [tuple(torch.as_tensor(m).double() for m in get(e)) for e in range(masters[0].shape[0])]
    out = []
    for e in range(masters[0].shape[0]):
        mats = [m[e] for m in masters]
        s = quant.scale(quant.expert_absmax(mats), bits[e])
        out.append(tuple(quant.codes(m, s, bits[e]).double() * s for m in mats))
    return out


def reference(x, ids, g, residual, experts):
    x = x.double()
    y = torch.zeros_like(x) if residual is None else residual.double()
    for e, (w1, w3, w2) in enumerate(experts):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        a = x[t] @ w1.t()
        h = a * torch.sigmoid(a) * (x[t] @ w3.t())
        y.index_add_(0, t, (h @ w2.t()) * g[t, j].double()[:, None])
    return y


def compare(y, ref, what):
    bf16 = y.dtype == torch.bfloat16
    d, ref = y.detach().cpu().double() - ref, ref
    rn, mx = float(ref.norm()), float(ref.abs().max())
    if mx == 0.0:
        assert float(d.abs().max()) == 0.0, what
        return
    log(f"  {what}: normwise {float(d.norm()) / rn:.2e} max {float(d.abs().max()) / mx:.2e}")
    assert float(d.norm()) / rn <= YTOL_NORM + (2.0 ** -8 if bf16 else 0.0), what
    assert float(d.abs().max()) / mx <= YTOL_MAX + (2.0 ** -8 if bf16 else 0.0), what


def routes(T, E, k, seed, skewed=False):
    gen = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=gen)
    if skewed:
        z[:, 0] += 20.0
        z[: T // 2, 1] += 10.0
    ids = z.topk(k, dim=1)[1].to(torch.int32)
    g = torch.rand(T, k, generator=gen) + 0.1
    return ids, g


CASES = [
    # name, shape, T, layout, skewed
    ("own_T1", dict(E=8, d=256, F=512, k=2), 1, "eq2", False),
    ("own_T12", dict(E=8, d=256, F=512, k=2), 12, "eq2", False),
    ("own_all_experts", dict(E=16, d=128, F=256, k=16), 9, "eq2", False),
    ("streaming_T40", dict(E=32, d=256, F=384, k=2), 40, "eq2", False),
    ("streaming_skewed_T150", dict(E=16, d=256, F=384, k=2), 150, "eq2", True),
    ("streaming_E80_T5", dict(E=80, d=128, F=128, k=32), 5, "eq2", False),
    ("bitplane_T24", dict(E=8, d=256, F=384, k=2), 24, "bitplane", False),
    ("bitplane_T6", dict(E=8, d=256, F=384, k=2), 6, "bitplane", False),
    ("matrix_core_T600", dict(E=8, d=512, F=384, k=2), 600, "eq2", False),
    ("matrix_core_T2500", dict(E=8, d=256, F=128, k=2), 2500, "eq2", True),
]


def build(name, shape, T, layout):
    wl = synth.WORKLOADS["decode_fine"].scaled(name=f"routed_{name}", T=T, **shape)
    masters = synth.expert_weights(wl)
    layer, _ = make_layer(wl, masters, max_tokens=T, layout=layout)
    bits = [(3, 4, 8)[e % 3] for e in range(wl.E)] if layout == "eq2" else [1 + e % 8 for e in range(wl.E)]
    layer.quantize_experts(bits)
    return wl, layer, weights64(masters, bits, layout)


@pytest.mark.parametrize("name,shape,T,layout,skewed", CASES, ids=[c[0] for c in CASES])
def test_given_routes(name, shape, T, layout, skewed):
    wl, layer, experts = build(name, shape, T, layout)
    x, logits = synth.tokens(wl, T=T)
    xd = x.cuda()
    gen = torch.Generator().manual_seed(T)
    res = torch.randn(T, wl.d, generator=gen)
    ids, g = routes(T, wl.E, wl.k, T, skewed)
    log(f"routed {name}")
    plain = layer.moe_forward(xd, logits.cuda())

    def call(ids, g, residual=None, **kw):
        return layer.moe_forward_routed(xd, ids.cuda(), g.cuda(), None if residual is None else residual.cuda(), **kw)

    compare(call(ids, g), reference(x, ids, g, None, experts), "fp32")
    compare(call(ids, g, res), reference(x, ids, g, res, experts), "fp32 + residual")
    r16 = res.bfloat16()
    compare(call(ids, g, r16), reference(x, ids, g, r16, experts), "bf16 + residual")
    compare(call(ids, g, out_dtype=torch.bfloat16), reference(x, ids, g, None, experts), "bf16")
    # the residual's own buffer
    y = r16.cuda()
    assert layer.moe_forward_routed(xd, ids.cuda(), g.cuda(), y, y=y) is y
    compare(y, reference(x, ids, g, r16, experts), "in place")
    # slots without an expert (-1 and ids that name none), their weights not
    # finite; whole tokens without; one expert named twice
    ids2, g2 = ids.clone(), g.clone()
    ids2[::3, 0] = -1
    g2[::3, 0] = float("nan")
    if wl.k > 1:
        ids2[1::4, 1] = wl.E + 5
        g2[1::4, 1] = float("inf")
        ids2[2::5, 1] = ids2[2::5, 0]
    if T > 4:
        ids2[4] = -7
    # (a token whose second slot names its first one's expert again, with an
    # infinite weight, has no finite result; every other token does)
    want = reference(x, ids2, g2, r16, experts)
    got = call(ids2, g2, r16)
    fine = want.isfinite().all(dim=1)
    infinite = ((ids2 >= 0) & (ids2 < wl.E) & ~g2.isfinite()).any(dim=1)
    assert torch.equal(fine, ~infinite)
    assert bool((~got.isfinite()).any(dim=1)[~fine.cuda()].all())
    compare(got[fine.cuda()], want[fine], "slots without an expert")
    if T > 4:
        assert torch.equal(got[4].cpu(), r16[4])
    # nothing at all, after a batch that had experts
    none = torch.full_like(ids, -1)
    assert torch.equal(call(none, g, r16).cpu(), r16)
    assert float(call(none, g).abs().max()) == 0.0
    # a smaller batch after a larger one, and the other forward untouched
    if T > 2:
        compare(layer.moe_forward_routed(xd[:2], ids[:2].cuda(), g[:2].cuda()), reference(x[:2], ids[:2], g[:2], None, experts), "2 tokens")
    again = layer.moe_forward(xd, logits.cuda())
    assert torch.equal(plain, again)


def test_routes_of_the_router_give_the_same_forward():
    """pw_route's ids and weights through pw_moe_forward_routed against
    pw_moe_forward on the logits: the same kernels on the same pairs. Equal
    up to the fp32 sums' order (experts take their tokens in any order, which
    no sum sees; the gate/up kernel may route itself with other K splits)."""
    wl, layer, _ = build("same", dict(E=32, d=256, F=384, k=4), 50, "eq2")
    x, logits = synth.tokens(wl, T=50)
    ids, g, _ = layer.route(logits.cuda())
    a = layer.moe_forward(x.cuda(), logits.cuda())
    b = layer.moe_forward_routed(x.cuda(), ids, g)
    torch.cuda.synchronize()
    assert float((a - b).abs().max()) <= 2.0 ** -20 * float(a.abs().max())


@pytest.mark.parametrize("name,shape,T,layout", [c[:4] for c in CASES if c[0] in ("own_T12", "streaming_T40", "bitplane_T24", "matrix_core_T600")],
                         ids=["own_T12", "streaming_T40", "bitplane_T24", "matrix_core_T600"])
def test_captured_routed_forward_replays(name, shape, T, layout):
    """Replays with new routes, other eager forwards on the same workspace in
    between."""
    wl, layer, _ = build("graph_" + name, shape, T, layout)
    x, logits = synth.tokens(wl, T=T)
    xd, ld = x.cuda(), logits.cuda()
    sets = [routes(T, wl.E, wl.k, s, skewed=s == 2) for s in range(4)]
    sets[3][0][1::2] = -1
    ids, g = (t.cuda() for t in sets[0])
    res = torch.randn(T, wl.d, device="cuda").bfloat16()
    want_plain = layer.moe_forward(xd, ld)
    layer.moe_forward_routed(xd, ids, g, res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.moe_forward_routed(xd, ids, g, res)
    for i, w in enumerate(sets[1:] + sets[:1]):
        ids.copy_(w[0].cuda())
        g.copy_(w[1].cuda())
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(layer.moe_forward(xd, ld), want_plain), i
        eager = layer.moe_forward_routed(xd, ids, g, res)
        torch.cuda.synchronize()
        assert torch.equal(got, eager), i


def test_a_graph_captured_first_and_not_replayed():
    """A capture before any other call leaves nothing behind: the eager call
    after it, the graph's replay after that, and calls between replays with
    other batch sizes all count from zero."""
    wl, layer, experts = build("capture_first", dict(E=32, d=256, F=384, k=2), 40, "eq2")
    x, _ = synth.tokens(wl, T=40)
    xd = x.cuda()
    ids, g = routes(40, wl.E, wl.k, 1)
    i, w = ids.cuda(), g.cuda()
    torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(0x7f)
    layer.bind_workspace(torch.full((layer.workspace_bytes(),), 0x7f, dtype=torch.uint8, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.moe_forward_routed(xd, i, w)
    want = reference(x, ids, g, None, experts)
    compare(layer.moe_forward_routed(xd, i, w), want, "eager after the capture")
    for n in (40, 17, 3):
        graph.replay()
        torch.cuda.synchronize()
        compare(y, want, "replay")
        compare(layer.moe_forward_routed(xd[:n], i[:n], w[:n]), reference(x[:n], ids[:n], g[:n], None, experts), f"eager {n}")


def test_given_routes_with_a_host_tier():
    wl, layer, experts = build("tier", dict(E=16, d=256, F=384, k=2), 40, "eq2")
    x, _ = synth.tokens(wl, T=40)
    ids, g = routes(40, wl.E, wl.k, 1)
    want = layer.moe_forward_routed(x.cuda(), ids.cuda(), g.cuda())
    layer.alloc_host_tier(16 * layer.slot_bytes())
    layer.alloc_pool(5 * layer.slot_bytes())
    layer.quantize_experts([(3, 4, 8)[e % 3] for e in range(wl.E)])
    for _ in range(2):
        got = layer.moe_forward_routed(x.cuda(), ids.cuda(), g.cuda())
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    ids[:] = 3
    ids[:, 1] = -1
    got = layer.moe_forward_routed(x.cuda(), ids.cuda(), g.cuda())
    compare(got, reference(x, ids, g, None, experts), "host tier")
    assert layer.residency()[0][3] >= 0


def test_no_tokens():
    wl, layer, _ = build("none", dict(E=8, d=128, F=128, k=2), 4, "eq2")
    y = layer.moe_forward_routed(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"),
                                 torch.empty(0, 2, dtype=torch.int32, device="cuda"), torch.empty(0, 2, device="cuda"))
    assert y.shape == (0, 128)


@pytest.mark.parametrize("T", [1, 48, 700])
def test_moe_block(T):
    """Router logits, gated routing, shared expert, routed experts and the
    residual as one block, against the float64 block on the ids it chose
    (the choice itself is the gate's own test); shared expert and residual
    are rounded to bf16 on the way (one more half step each)."""
    from mixed_precision_weight_page_amd import linear
    wl, layer, experts = build(f"block{T}", dict(E=16, d=256, F=384, k=4), T, "eq2")
    gen = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    x = rand(T, 256).bfloat16()
    gate_w = (rand(16, 256) / 16).bfloat16()
    up, down = (rand(2 * 200, 256) / 16).bfloat16(), (rand(256, 200) / 14).bfloat16()
    res, bias = rand(T, 256).bfloat16(), rand(16) * 0.1
    mask = torch.ones(T, dtype=torch.bool)
    mask[T // 2:T // 2 + 1] = T == 1
    kw = dict(score="sigmoid", bias=bias.cuda(), n_group=4, topk_group=2, group_score="top2", renorm=True, scale=2.5, mask=mask.cuda())
    args = dict(shared=(up.cuda(), down.cuda()), residual=res.cuda())
    y, ids, g, counts = layer.moe_block(x.cuda(), gate_w.cuda(), **args, **kw)
    logits = linear(x.cuda(), gate_w.cuda(), out_dtype=torch.float32)
    ids2, g2, counts2 = layer.route_gated(logits, **kw)
    assert torch.equal(ids, ids2) and torch.equal(g, g2) and torch.equal(counts, counts2)
    assert int(counts.sum()) == int((ids >= 0).sum()) == 4 * int(mask.sum())
    xd = x.double()
    z = xd @ up.double().t()
    h = z[:, :200] * torch.sigmoid(z[:, :200]) * z[:, 200:]
    shared = h @ down.double().t() + res.double()
    ref = reference(x, ids.cpu(), g.cpu(), shared, experts)
    d = y.cpu().double() - ref
    # bf16: h, the shared sum and y are rounded
    assert float(d.norm() / ref.norm()) <= YTOL_NORM + 3 * 2.0 ** -8
    assert float(d.abs().max() / ref.abs().max()) <= YTOL_MAX + 3 * 2.0 ** -8
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, *_ = layer.moe_block(x.cuda(), gate_w.cuda(), **args, **kw, stream=side)
    side.synchronize()
    assert torch.equal(y, y2)
