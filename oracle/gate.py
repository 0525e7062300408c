"""Oracle of gated routing: scores, groups, biased top-k choice, weights.

TEST INFRASTRUCTURE: imported only by tests; never by the GPU library. Plain
float64 Python over one token at a time, written from the definition:

* an expert is to be had unless its logit is NaN, -inf or the lowest finite
  value of the logits' type;
* s = softmax over the experts to be had, or 1 / (1 + e^-l); c = s + bias;
* the topk_group best groups of consecutive experts stay (score: the largest
  c, or the sum of the two largest; ties: lower group);
* the k largest c among them are chosen (ties: lower expert; c NaN or -inf:
  not chosen); weight scale * s, renormalised over the chosen if asked.
"""
from __future__ import annotations

import math


def _scores(l, ok, score):
    """log s of every expert (-inf where not to be had); infinite logits by their limits."""
    out = [-math.inf] * len(l)
    live = [e for e in range(len(l)) if ok[e]]
    if not live:
        return out
    if score == "softmax":
        m = max(l[e] for e in live)
        z = [0.0 if l[e] == m else l[e] - m for e in live]
        total = math.log(math.fsum(math.exp(v) for v in z))
        for e, v in zip(live, z):
            out[e] = v - total
    else:
        for e in live:
            x = l[e]
            out[e] = min(x, 0.0) - math.log1p(math.exp(-abs(x))) if math.isfinite(x) else 0.0
    return out


def token(l, lowest, k, score="softmax", bias=None, n_group=1, topk_group=1, top2=False, renorm=False, scale=1.0,
          live=True):
    """(ids, weights) of one token; l a list of floats."""
    E = len(l)
    ok = [live and not math.isnan(v) and v > lowest for v in l]
    logs = _scores(l, ok, score)
    c = [-math.inf] * E
    for e in range(E):
        if ok[e]:
            # without a bias the order is the logits' (scores may round to one value)
            v = math.exp(logs[e]) + (bias[e] if bias is not None else 0.0)
            c[e] = -math.inf if math.isnan(v) else v
    order_by_logit = bias is None
    key = [(l[e] if order_by_logit else c[e]) if c[e] > -math.inf else -math.inf for e in range(E)]
    gs = E // n_group
    if n_group > 1:
        groups = []
        for q in range(n_group):
            part = sorted((c if top2 else key)[q * gs:(q + 1) * gs], reverse=True)
            s = part[0]
            if top2 and gs > 1 and part[1] > -math.inf:
                s += part[1]
            groups.append(s)
        stay = set(sorted(range(n_group), key=lambda q: (-groups[q], q))[:topk_group])
        key = [key[e] if e // gs in stay else -math.inf for e in range(E)]
    chosen = [e for e in sorted(range(E), key=lambda e: (-key[e], e)) if key[e] > -math.inf][:k]
    if renorm and chosen:
        top = max(logs[e] for e in chosen)
        if top > -math.inf:
            w = [math.exp(logs[e] - top) for e in chosen]
            w = [v / math.fsum(w) * scale for v in w]
        else:
            w = [0.0] * len(chosen)
    else:
        w = [math.exp(logs[e]) * scale for e in chosen]
    return chosen + [-1] * (k - len(chosen)), w + [0.0] * (k - len(chosen))


def route(logits, lowest, k, mask=None, **kw):
    """Rows of (ids, weights) and the pairs per expert."""
    rows = [token([float(v) for v in row], lowest, k, live=mask is None or bool(mask[t]), **kw)
            for t, row in enumerate(logits)]
    counts = [0] * (len(logits[0]) if len(logits) else 0)
    for ids, _ in rows:
        for e in ids:
            if e >= 0:
                counts[e] += 1
    return [r[0] for r in rows], [r[1] for r in rows], counts
