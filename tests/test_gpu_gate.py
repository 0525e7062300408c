"""GPU tests of pw_route_gated against the float64 oracle (oracle/gate.py):
ids and counts exactly, weights within 2^-20 of the value: the logit's
difference to the largest rounds by half an ulp of at most 32 (2^-19 / 2
relative after the exponential for logits within 32 of each other), the
exponential, sum and quotient by a few 2^-24 more. Logits are drawn within
that range; the tests of extreme logits say their own bound."""
import math

import pytest
import torch

from layer_cases import log
from oracle import gate as gate_oracle

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
WTOL = 2.0 ** -20 + 2.0 ** -20   # exponent's rounding, and the rest


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(E, k, T):
    from mixed_precision_weight_page_amd import PagedMoELayer
    return PagedMoELayer(E, 128, 128, k, max_tokens=max(T, 1))


def draw(T, E, dtype, seed, cols=0):
    g = torch.Generator().manual_seed(seed)
    buf = (torch.randn(T, E + cols, generator=g) * 2.0).clamp_(-16, 16).to(dtype)
    return buf[:, :E], (torch.randn(E, generator=g) * 0.1)


def check(layer, logits, wtol=WTOL, **kw):
    """logits on the CPU, possibly strided; kw as route_gated's, tensors on the CPU."""
    buf = logits
    if logits.stride(0) != logits.shape[1] and logits.shape[0] > 1:
        full = torch.full((logits.shape[0], logits.stride(0)), float("nan"), dtype=logits.dtype)
        full[:, :logits.shape[1]] = logits
        buf = full.cuda()[:, :logits.shape[1]]
    else:
        buf = logits.cuda()
    dev = {n: (v.cuda() if isinstance(v, torch.Tensor) else v) for n, v in kw.items()}
    ids, g, counts = layer.route_gated(buf, **dev)
    torch.cuda.synchronize()
    compare(layer, logits, ids, g, counts, wtol, **kw)
    return ids, g, counts


def group_gap(l, low, score, bias, n_group, topk_group):
    """Relative gap between the sums of the last group that stays and the
    first that goes; infinite if they hold the same two logits and biases (a
    tie in any arithmetic) or one of them has none."""
    E = len(l)
    ok = [v > low for v in l]
    logs = gate_oracle._scores(l, ok, score)
    b = [0.0] * E if bias is None else bias.double().tolist()
    gs = E // n_group
    sums = []
    for q in range(n_group):
        best = sorted(((math.exp(logs[e]) + b[e], l[e], b[e]) for e in range(q * gs, (q + 1) * gs) if ok[e]), reverse=True)[:2]
        sums.append((sum(v[0] for v in best) if best else -math.inf, -q, sorted(v[1:] for v in best)))
    sums.sort(reverse=True)
    if topk_group >= n_group:
        return math.inf
    x, y = sums[topk_group - 1], sums[topk_group]
    if x[2] == y[2] or not x[2] or not y[2] or not math.isfinite(x[0] - y[0]):
        return math.inf
    return (x[0] - y[0]) / max(abs(x[0]), 1e-300)


def compare(layer, logits, ids, g, counts, wtol=WTOL, score="softmax", bias=None, n_group=1, topk_group=1,
            group_score="max", renorm=False, scale=1.0, mask=None):
    low = float(torch.finfo(logits.dtype).min)
    want_ids, want_g, want_counts = gate_oracle.route(
        logits.double().tolist(), low, layer.k, mask=None if mask is None else mask.tolist(), score=score,
        bias=None if bias is None else bias.double().tolist(), n_group=n_group, topk_group=topk_group,
        top2=group_score == "top2", renorm=renorm, scale=scale)
    want = torch.tensor(want_ids, dtype=torch.int32).reshape(ids.shape)
    decided = torch.ones(ids.shape[0], dtype=torch.bool)
    if n_group > 1 and group_score == "top2":
        # Two group sums can be nearer than fp64 can tell: a score is off by
        # at most 10 2^-53 in the oracle (the exponential of a logarithm of
        # magnitude up to 8) and 6 2^-53 in the kernel (exponential, sum,
        # quotient, bias), so sums S and S' of different experts' scores with
        # |S - S'| <= 2 (10 + 6) 2^-53 S = 2^-48 S may come in either order.
        decided = torch.tensor([group_gap(row, low, score, bias, n_group, topk_group) > 2.0 ** -48
                                for row in logits.double().tolist()], dtype=torch.bool)
    off = (ids.cpu() != want).any(dim=1) & decided
    assert not bool(off.any()), f"token {int(off.nonzero()[0])} of {int(off.sum())}"
    if not bool(decided.all()):
        log(f"  {int((~decided).sum())} tokens whose groups fp64 cannot tell apart")
        ids, g, counts = ids.cpu()[decided], g.cpu()[decided], None
        want_g = [w for w, d in zip(want_g, decided.tolist()) if d]
    wg = torch.tensor(want_g, dtype=torch.float64).reshape(g.shape)
    err = (g.cpu().double() - wg).abs()
    assert bool((err <= wtol * wg.abs() + 1e-37).all()), float((err / wg.abs().clamp_min(1e-37)).max())
    if counts is not None:
        assert counts.cpu().tolist() == (want_counts or [0] * layer.E)


CASES = [
    # T, E, k, dtype, kw
    (1, 1, 1, "f32", {}),
    (1, 8, 2, "f32", dict(renorm=True)),
    (3, 5, 5, "bf16", dict(score="sigmoid", scale=2.5)),
    (16, 64, 6, "f16", dict(bias=True, renorm=True)),
    (17, 65, 8, "f32", dict(score="sigmoid", bias=True)),
    (64, 128, 8, "f32", {}),
    (65, 100, 7, "bf16", dict(bias=True, mask=True, cols=3)),
    (33, 256, 8, "f32", dict(score="sigmoid", bias=True, n_group=8, topk_group=4, group_score="top2", renorm=True, scale=2.5)),
    (40, 257, 32, "f32", dict(bias=True)),
    (9, 1024, 32, "bf16", dict(n_group=64, topk_group=3)),
    (20, 96, 4, "f32", dict(n_group=6, topk_group=2, group_score="top2")),
    (20, 60, 4, "f32", dict(n_group=20, topk_group=9, group_score="top2", score="sigmoid", bias=True)),
    (20, 64, 3, "f16", dict(n_group=64, topk_group=5, group_score="top2", score="sigmoid")),
    (18, 510, 10, "f32", dict(n_group=17, topk_group=5, group_score="top2", bias=True)),
    # past the batches that take a wave per token
    (1040, 16, 2, "f32", dict(renorm=True)),
    (1041, 40, 17, "bf16", dict(score="sigmoid", bias=True, cols=1)),
    (1100, 256, 8, "f32", dict(score="sigmoid", bias=True, n_group=8, topk_group=4, group_score="top2", renorm=True, scale=2.5)),
    (1030, 128, 32, "f16", dict(n_group=16, topk_group=7, mask=True)),
    (1030, 200, 5, "f32", dict(n_group=40, topk_group=9, group_score="top2", bias=True)),
    (1055, 30, 4, "bf16", dict(bias=True, n_group=2, topk_group=1)),
]


@pytest.mark.parametrize("T,E,k,dtype,kw", CASES, ids=[f"T{c[0]}_E{c[1]}_k{c[2]}_{c[3]}_{i}" for i, c in enumerate(CASES)])
def test_gate_matches_the_oracle(T, E, k, dtype, kw):
    kw = dict(kw)
    logits, bias = draw(T, E, DT[dtype], 7 * T + E, kw.pop("cols", 0))
    if kw.pop("bias", False):
        kw["bias"] = bias
    if kw.pop("mask", False):
        kw["mask"] = torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.7
    log(f"gate T={T} E={E} k={k} {dtype}")
    check(make(E, k, T), logits, **kw)


@pytest.mark.parametrize("T", [16, 17, 1100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_and_nearly_equal_scores(T, score):
    """Ties take the lower expert; scores that fp32 cannot tell apart are
    chosen by their fp64 values."""
    E, k = 64, 8
    layer = make(E, k, T)
    check(layer, torch.zeros(T, E), score=score)
    check(layer, torch.zeros(T, E), score=score, bias=torch.zeros(E), n_group=8, topk_group=3, group_score="top2")
    # neighbouring fp32 logits (their scores differ by less than an fp32 ulp
    # near 1), in a scattered order
    g = torch.Generator().manual_seed(5)
    step = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float()
    for base in (0.75, 6.0, -3.0):
        logits = torch.tensor(base) + step * 2.0 ** -21
        check(layer, logits, score=score, bias=torch.zeros(E))
        check(layer, logits, score=score, bias=torch.full((E,), 0.25), n_group=4, topk_group=2, group_score="top2", renorm=True)


@pytest.mark.parametrize("T", [5, 30, 1200])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_and_tokens_that_are_not_to_be_had(T, dtype, score):
    """-inf, the type's lowest value and NaN take an expert out; rows with
    fewer than k left, with none, and masked rows full of NaN; +inf."""
    E, k = 24, 6
    logits, bias = draw(T, E, DT[dtype], 11)
    logits = logits.clone()
    low = torch.finfo(DT[dtype]).min
    logits[:, 1], logits[:, 5], logits[:, 9] = -math.inf, low, math.nan
    logits[0] = -math.inf
    logits[1] = low
    logits[2] = math.nan
    logits[3, 4:] = -math.inf        # at most three left
    logits[4, 10] = math.inf
    if T > 20:
        logits[20, 3:7] = math.inf
    mask = torch.ones(T, dtype=torch.uint8)
    if T > 8:
        mask[7] = 0
        logits[7] = math.nan
    layer = make(E, k, T)
    b = bias.clone()
    b[2], b[3], b[6] = -math.inf, math.nan, math.inf
    for kw in (dict(), dict(renorm=True), dict(bias=bias), dict(bias=b, renorm=True),
               dict(bias=bias, n_group=4, topk_group=2, group_score="top2", renorm=True),
               dict(n_group=8, topk_group=3)):
        check(layer, logits, score=score, mask=mask, **kw)


def test_logits_far_apart():
    """Renormalised weights where every score underflows fp32, and scores
    that saturate: the logit difference rounds by half an ulp of up to 512
    (2^-15 relative after the exponential)."""
    for score in ("softmax", "sigmoid"):
        logits = torch.tensor([[-300.25, -301.5, -302.125, -303.0], [300.25, 301.5, 302.125, 299.0],
                               [80.0, -80.0, 0.0, 40.0], [-3e38, 3e38, 1e-40, -1e-40]])
        for renorm in (False, True):
            check(make(4, 3, 4), logits, wtol=2.0 ** -15, score=score, renorm=renorm)


def test_no_tokens_and_no_counts():
    layer = make(8, 2, 4)
    ids, g, counts = layer.route_gated(torch.empty(0, 8, device="cuda"))
    assert ids.shape == (0, 2) and counts.cpu().tolist() == [0] * 8
    logits, _ = draw(4, 8, torch.float32, 1)
    ids, g, counts = layer.route_gated(logits.cuda(), with_counts=False)
    assert counts is None
    compare(layer, logits, ids, g, None)


@pytest.mark.parametrize("T", [4, 70, 1500])
def test_captured_gate_replays(T):
    E, k = 64, 4
    layer = make(E, k, T)
    batches = [draw(T, E, torch.float32, s)[0] for s in range(4)]
    bias = draw(1, E, torch.float32, 9)[1].cuda()
    x = batches[0].cuda()
    kw = dict(score="sigmoid", bias=bias, n_group=8, topk_group=3, group_score="top2")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.route_gated(x, **kw)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.route_gated(x, **kw)
    for b in batches[1:]:
        x.copy_(b.cuda())
        for o in out:
            o.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        eager = layer.route_gated(b.cuda(), **kw)
        for o, e in zip(out, eager):
            assert torch.equal(o, e)


def test_another_stream():
    """Outputs of a call on a side stream, allocated for that stream, while
    the inputs are dropped at once."""
    E, k, T = 128, 8, 2000
    layer = make(E, k, T)
    logits, bias = draw(T, E, torch.float32, 3)
    side = torch.cuda.Stream()
    d, b = logits.cuda(), bias.cuda()
    side.wait_stream(torch.cuda.current_stream())
    ids, g, counts = layer.route_gated(d, bias=b, stream=side)
    del d, b
    junk = [torch.full((T, E), 1e9, device="cuda") for _ in range(4)]
    side.synchronize()
    compare(layer, logits, ids, g, counts, bias=bias)
    del junk
