"""GPU tests of the calls around the expert layer as a block uses them:
streams given by handle, captured and replayed blocks."""
import pytest
import torch

import synth
from layer_cases import YTOL_MAX, cpu_threads, log, make_layer
from test_gpu_linear import reference as linear_reference
from test_gpu_routed import reference, weights64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cpu_threads()


GATE = dict(score="sigmoid", n_group=4, topk_group=2, group_score="top2", renorm=True, scale=2.5)


class Block:
    """A layer of 16 experts with pages of every width, its router's and its
    shared expert's weights, and T tokens."""
    def __init__(self, T, seed=1, layout="eq2", **shape):
        wl = synth.WORKLOADS["decode_fine"].scaled(name="block", T=max(T, 1), **{**dict(E=16, d=256, F=384, k=4), **shape})
        self.wl = wl
        self.masters = synth.expert_weights(wl)
        self.layer, _ = make_layer(wl, self.masters, max_tokens=max(T, 1), layout=layout)
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


@pytest.mark.parametrize("T", [1, 48, 700])
def test_a_captured_block_replays(T):
    """Each replay, with new tokens, against the eager block bit for bit;
    eager blocks of other sizes between the replays."""
    b = Block(T)
    x, res = (t.clone() for t in b.batches[0])
    log(f"captured block T={T}")
    b(x, res)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b(x, res)
    for i, (nx, nr) in enumerate(b.batches[1:] + b.batches[:1]):
        x.copy_(nx)
        res.copy_(nr)
        for o in out:
            o.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        n = max(1, T // 3)
        small = b(nx[:n], nr[:n])
        assert bool(small[0].isfinite().all())
        for g, w in zip(got, b(nx, nr)):
            assert torch.equal(g, w), i


@pytest.mark.parametrize("layout", ["eq2", "bitplane"])
def test_two_graphs_of_one_layer(layout):
    """Two captured blocks share the layer's workspace; replayed in turn, and
    one twice in a row, each gives the eager block."""
    b = Block(60, layout=layout)
    xs = [b.batches[0][0].clone(), b.batches[1][0][:9].clone()]
    rs = [b.batches[0][1].clone(), b.batches[1][1][:9].clone()]
    for x, r in zip(xs, rs):
        b(x, r)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g, x, r in zip(graphs, xs, rs):
        with torch.cuda.graph(g):
            outs.append(b(x, r))
    keep = []
    for step, i in enumerate((0, 1, 1, 0, 0, 1)):
        xs[i].copy_(b.batches[step % 3][0][:xs[i].shape[0]])
        outs[i][0].fill_(float("nan"))
        graphs[i].replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs[i]]
        keep.append((i, xs[i].clone(), got))
        if step % 2:   # after every other replay the next one follows it directly
            for j, x, o in keep:
                for g, w in zip(o, b(x, rs[j])):
                    assert torch.equal(g, w), step
            keep = []


def test_captured_given_routes_with_a_host_tier():
    """Pages read through the device's cache of slots, decided at each replay
    on the device."""
    b = Block(40, k=2, d=256)
    x, _ = b.batches[0]
    gen = torch.Generator().manual_seed(3)
    sets = [(torch.randn(40, 16, generator=gen).topk(2, dim=1)[1].int().cuda(), torch.rand(40, 2, generator=gen).cuda()) for _ in range(4)]
    sets[2][0][:, :] = 5
    sets[3][0][::2] = -1
    want = [b.layer.moe_forward_routed(x, i, g) for i, g in sets]
    b.layer.alloc_host_tier(16 * b.layer.slot_bytes())
    b.layer.alloc_pool(5 * b.layer.slot_bytes())
    b.layer.quantize_experts(b.bits)
    ids, g = (t.clone() for t in sets[0])
    assert torch.equal(b.layer.moe_forward_routed(x, ids, g), want[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.layer.moe_forward_routed(x, ids, g)
    for n in (1, 2, 3, 0, 1):
        ids.copy_(sets[n][0])
        g.copy_(sets[n][1])
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[n]), n
        assert torch.equal(b.layer.moe_forward_routed(x, *sets[3]), want[3])


PATHS = [("own", 9, "eq2"), ("streaming", 40, "eq2"), ("bitplane", 40, "bitplane"), ("matrix_core", 700, "eq2")]


@pytest.mark.parametrize("name,T,layout", PATHS, ids=[p[0] for p in PATHS])
def test_what_tokens_without_experts_hold_does_not_matter(name, T, layout):
    """Padded tokens (every id -1) may hold NaN and infinities: their rows
    are the residual's, the others as with zeros there."""
    b = Block(T, layout=layout)
    x, res = b.batches[0]
    gen = torch.Generator().manual_seed(T)
    ids = torch.randn(T, 16, generator=gen).topk(4, dim=1)[1].int().cuda()
    g = torch.rand(T, 4, generator=gen).cuda()
    gone = torch.zeros(T, dtype=torch.bool, device="cuda")
    gone[1::3] = True
    ids[gone] = -1
    g[gone] = float("nan")
    clean, dirty = x.clone(), x.clone()
    clean[gone] = 0.0
    dirty[gone] = float("nan")
    dirty[1] = float("inf")
    a = b.layer.moe_forward_routed(clean, ids, g, res)
    c = b.layer.moe_forward_routed(dirty, ids, g, res)
    assert torch.equal(a, c) and torch.equal(c[gone], res[gone]) and bool(c.isfinite().all())


@pytest.mark.parametrize("name,T,layout", PATHS, ids=[p[0] for p in PATHS])
def test_the_tokens_own_rows_as_residual_and_output(name, T, layout):
    """y and residual may be x: the sums are added last, after every expert
    has read its tokens."""
    b = Block(T, layout=layout)
    x, _ = b.batches[0]
    gen = torch.Generator().manual_seed(T)
    ids = torch.randn(T, 16, generator=gen).topk(4, dim=1)[1].int().cuda()
    g = torch.rand(T, 4, generator=gen).cuda()
    want = b.layer.moe_forward_routed(x, ids, g, residual=x)
    inside = x.clone()
    assert b.layer.moe_forward_routed(inside, ids, g, residual=inside, y=inside) is inside
    assert torch.equal(inside, want)


@pytest.mark.parametrize("name,T,layout", PATHS, ids=[p[0] for p in PATHS])
def test_every_slot_with_the_same_expert(name, T, layout):
    """An expert named by all slots of every token counts with the sum of the
    weights: as named once with that sum (quarters of whole numbers: exact)."""
    b = Block(T, layout=layout)
    x, _ = b.batches[0]
    ids = torch.full((T, 4), 7, dtype=torch.int32, device="cuda")
    g = (torch.randint(1, 9, (T, 4), generator=torch.Generator().manual_seed(T)).float() / 4).cuda()
    once, total = torch.full_like(ids, -1), torch.zeros_like(g)
    once[:, 0], total[:, 0] = 7, g.sum(dim=1)
    assert torch.equal(b.layer.moe_forward_routed(x, ids, g), b.layer.moe_forward_routed(x, once, total))


@pytest.mark.parametrize("T", [1, 48, 700])
def test_a_block_in_fp32_keeps_the_shared_sum(T):
    """With an fp32 residual and output only the shared expert's SwiGLU rows
    are rounded on the way, to bf16 (half a step, 2^-8 of each; the products
    around it within the dense product's bounds); the routed experts have the
    layer's tolerance, per element of their largest. The residual is large,
    so that a rounding of the sum to bf16 would go far past that."""
    b = Block(T)
    x, res = b.batches[0]
    res = res.float() * 1000.0
    y, ids, g, _ = b(x, res, out_dtype=torch.float32)
    assert y.dtype == torch.float32
    up, down = (w.cpu() for w in b.shared)
    h, dh = linear_reference(x.cpu(), up, None, "swiglu", None)
    dh = dh + 2.0 ** -8 * (h.abs() + dh)
    S = (h.abs() + dh) @ down.double().abs().t()
    routed = reference(x.cpu(), ids.cpu(), g.cpu(), None, weights64(b.masters, b.bits, "eq2"))
    want = res.cpu().double() + h @ down.double().t() + routed
    tol = dh @ down.double().abs().t() + (200 + 2) * 2.0 ** -23 * S + YTOL_MAX * routed.abs().max() + 2 * 2.0 ** -24 * (want.abs() + S)
    err = (y.cpu().double() - want).abs()
    log(f"block in fp32 T={T}: {float((err / tol).max()):.2f} of the bound, a rounding to bf16 {float((2.0 ** -8 * want.abs() / tol).max()):.0f}")
    assert bool((err <= tol).all())


def test_a_block_without_tokens():
    b = Block(0)
    x, res = b.batches[0]
    y, ids, g, counts = b(x, res)
    assert y.shape == (0, 256) and ids.shape == g.shape == (0, 4) and counts.cpu().tolist() == [0] * 16


@pytest.mark.parametrize("name,T,layout", PATHS, ids=[p[0] for p in PATHS])
def test_given_routes_while_forwards_are_timed(name, T, layout):
    """pw_profile counts and times these forwards too, and changes none."""
    b = Block(T, layout=layout)
    x, res = b.batches[0]
    ids = torch.randn(T, 16, generator=torch.Generator().manual_seed(T)).topk(4, dim=1)[1].int().cuda()
    g = torch.full((T, 4), 0.25, device="cuda")
    want = b.layer.moe_forward_routed(x, ids, g, res)
    b.layer.profile(True)
    for _ in range(3):
        assert torch.equal(b.layer.moe_forward_routed(x, ids, g, res), want)
    times = b.layer.profile_read()
    b.layer.profile(False)
    assert times["forwards"] == 3
    assert all(times[n] > 0.0 for n in ("route_ms", "gate_up_ms", "down_ms", "combine_ms")), times
