"""GPU tests of pw_route_gated's choice bias where it is no ordinary number
(NaN, -inf, +inf) and scores tie, so that the choice is made again from fp64
scores. Logits take a few values only: choice scores are equal or far apart,
so the oracle's ids and counts have to be met exactly; weights as in
test_gpu_gate.py (logits within 32 of each other)."""
import math

import pytest
import torch

from layer_cases import log
from oracle import gate as gate_oracle

pytestmark = pytest.mark.gpu

LOW = float(torch.finfo(torch.float32).min)
WTOL = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(layer, logits, **kw):
    """logits and tensors of kw on the CPU; kw as route_gated's."""
    dev = {n: (v.cuda() if isinstance(v, torch.Tensor) else v) for n, v in kw.items()}
    ids, g, counts = layer.route_gated(logits.cuda(), **dev)
    opt = dict(kw, bias=None if kw.get("bias") is None else kw["bias"].double().tolist())
    opt["top2"] = opt.pop("group_score", "max") == "top2"
    want_ids, want_g, want_counts = gate_oracle.route(logits.double().tolist(), LOW, layer.k, **opt)
    want = torch.tensor(want_ids, dtype=torch.int32)
    off = (ids.cpu() != want).any(dim=1)
    assert not bool(off.any()), (int(off.nonzero()[0]), ids[off.cuda()][0].tolist(), want[off][0].tolist(), kw)
    wg = torch.tensor(want_g, dtype=torch.float64)
    assert bool(((g.cpu().double() - wg).abs() <= WTOL * wg.abs()).all())
    assert counts.cpu().tolist() == want_counts


def tied(T, E, seed):
    """Logits 0, 1 and 2 in random places: sums of two scores too are equal or
    differ by a twentieth of themselves."""
    return torch.randint(0, 3, (T, E), generator=torch.Generator().manual_seed(seed)).float()


# one token per 64 lanes in one workgroup and in several, per 16 lanes in one
# and in several
@pytest.mark.parametrize("T", [1, 16, 30, 70, 1100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_bias_of_nan_among_equal_scores(T, score):
    from mixed_precision_weight_page_amd import PagedMoELayer
    for E, k in ((4, 2), (24, 6), (64, 8)):
        layer = PagedMoELayer(E, 128, 128, k, max_tokens=T)
        bias = torch.zeros(E)
        bias[1] = math.nan
        bias[E - 1] = -math.inf
        log(f"NaN bias T={T} E={E} {score}")
        for logits in (torch.zeros(T, E), tied(T, E, T + E)):
            check(layer, logits, score=score, bias=bias)
            check(layer, logits, score=score, bias=bias, n_group=2, topk_group=2, renorm=True)
            if E > 4:
                for by in ("max", "top2"):
                    check(layer, logits, score=score, bias=bias, n_group=4, topk_group=2, group_score=by, renorm=True)


@pytest.mark.parametrize("T", [1, 16, 30, 70, 1100])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_with_one_and_with_two_infinite_scores_are_equal(T, score):
    """A group's sum is infinite with one c of +inf as with two: the lower
    group stays."""
    from mixed_precision_weight_page_amd import PagedMoELayer
    for E, n_group, k, at in ((16, 4, 2, (1, 4, 5)), (64, 8, 5, (9, 16, 23, 63)), (256, 8, 8, (40, 64, 95, 255))):
        layer = PagedMoELayer(E, 128, 128, k, max_tokens=T)
        bias = torch.zeros(E)
        bias[list(at)] = math.inf
        log(f"infinite bias T={T} E={E} {score}")
        for logits in (torch.zeros(T, E), tied(T, E, T + E)):
            for topk_group in (1, 2):
                for by in ("max", "top2"):
                    check(layer, logits, score=score, bias=bias, n_group=n_group, topk_group=topk_group, group_score=by)


@pytest.mark.parametrize("T", [1, 30, 1100])
def test_scores_that_fp64_rounds_to_one_value(T):
    """Sigmoid scores of logits above 37 are 1 and softmax scores 800 below
    the largest logit's 0 in fp64: without a bias the logits order them, with
    one of zeros they tie."""
    from mixed_precision_weight_page_amd import PagedMoELayer
    layer = PagedMoELayer(8, 128, 128, 4, max_tokens=T)
    for score, row in (("sigmoid", [40.0, 50.0, 38.0, 0.0, 45.0, 60.0, -1.0, 39.0]),
                       ("softmax", [0.0, -900.0, -800.0, 1.0, -850.0, -825.0, 2.0, -875.0])):
        logits = torch.tensor([row] * T)
        for bias in (None, torch.zeros(8)):
            ids, _, _ = layer.route_gated(logits.cuda(), score=score, bias=None if bias is None else bias.cuda())
            want, _ = gate_oracle.token(row, LOW, 4, score=score, bias=None if bias is None else [0.0] * 8)
            log(f"  {score} {'no bias' if bias is None else 'zeros'}: {want}")
            assert ids.cpu().tolist() == [want] * T
            live = sorted(range(8), key=lambda e: (-row[e], e)) if bias is None else None
            assert live is None or want == live[:4]
        tied = [e for e in range(8) if row[e] > 37] if score == "sigmoid" else [6, 3, 0, 1]
        assert want == tied[:4]


@pytest.mark.parametrize("T", [1, 16, 30, 70, 1100])
def test_softmax_beside_an_infinite_logit_that_is_not_chosen(T):
    """Its score is 1 and every other 0: the weights of the others are 0,
    renormalised as well (a sum of 0 gives weights of 0). Where it is chosen
    it has all the weight."""
    from mixed_precision_weight_page_amd import PagedMoELayer
    for E, k in ((8, 3), (96, 8)):
        layer = PagedMoELayer(E, 128, 128, k, max_tokens=T)
        logits = tied(T, E, T + E)
        logits[:, 5] = math.inf
        for b5 in (0.0, -4.0, -math.inf, math.nan):
            bias = torch.zeros(E)
            bias[5] = b5
            for renorm in (False, True):
                check(layer, logits, bias=bias, renorm=renorm, scale=2.5)
                check(layer, logits, bias=bias, renorm=renorm, n_group=2, topk_group=2)
                check(layer, logits, renorm=renorm)
