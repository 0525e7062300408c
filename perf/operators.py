"""The operators around the expert layer, as cases to measure and compare.

Three operators of a mixture-of-experts block in serving:

* ``route``   scores, groups, biased top-k choice and weights of the experts of each token
* ``linear``  a dense product with bias, activation and residual: the router's own logits, the always-on (shared) expert
* ``experts`` the products of the routed experts from quantized pages, given ids and weights, added to a residual

Where ``own`` is false, ``run`` computes them in plain torch operations; where it is true, with the package's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- cases

def _route(T, E, k, score="softmax", dtype="f32", groups=1, keep=1, group_score="max", bias=False, renorm=True,
           scale=1.0, padded=0.0, absent=0.0, pad_cols=0, name=None):
    c = dict(op="route", T=T, E=E, k=k, score=score, dtype=dtype, groups=groups, keep=keep, group_score=group_score,
             bias=bias, renorm=renorm, scale=scale, padded=padded, absent=absent, pad_cols=pad_cols)
    return dict(c, name=name) if name else c


def _linear(M, N, K, act="none", dtype="bf16", out="bf16", bias=False, residual=False, pad=0, name=None):
    c = dict(op="linear", M=M, N=N, K=K, act=act, dtype=dtype, out=out, bias=bias, residual=residual, pad=pad)
    return dict(c, name=name) if name else c


def _experts(T, E, d, F, k, bits="mixed", skew=0.0, padded=0.0, residual=True, name=None):
    c = dict(op="experts", T=T, E=E, d=d, F=F, k=k, bits=bits, skew=skew, padded=padded, residual=residual)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a single stream: launch latency; 256 experts in 8 groups, 4 kept, chosen by biased sigmoid scores
        _route(1, 256, 8, "sigmoid", groups=8, keep=4, group_score="top2", bias=True, scale=2.5, name="route_one_token"),
        # the decode batch of the 128-expert layer: softmax over all experts
        _route(64, 128, 8, renorm=False, name="route_decode"),
        # a padded batch of odd length whose logits come in bf16 from a wider buffer, some experts not to be had
        _route(1003, 64, 6, "softmax", "bf16", bias=True, padded=0.2, absent=0.1, pad_cols=3, name="route_ragged"),
        # a long prompt over 256 grouped experts
        _route(16384, 256, 8, "sigmoid", groups=8, keep=4, group_score="top2", bias=True, scale=2.5, name="route_prompt"),
        # the router's logits of the 128-expert decode batch: few columns, fp32 out
        _linear(64, 128, 2048, out="f32", bias=True, name="linear_router_logits"),
        # shared expert, 16 tokens: gate and up in one pass over the weights (d 4096, d_ff 14336)
        _linear(16, 14336, 4096, "swiglu", name="linear_shared_up_decode"),
        # shared expert's down product for one token, added to the residual stream
        _linear(1, 4096, 14336, residual=True, name="linear_shared_down_one"),
        # shared expert of a 4096-token prompt (d 4096, d_ff 1408)
        _linear(4096, 1408, 4096, "swiglu", name="linear_shared_up_prompt"),
        # odd everything: sizes no tile divides, rows of unaligned length, fp16
        _linear(777, 1001, 700, "gelu", "f16", "f16", bias=True, residual=True, pad=5, name="linear_odd"),
        # a square-ish dense layer over a long prompt
        _linear(8192, 4096, 4096, "gelu_tanh", bias=True, residual=True, name="linear_prompt"),
        # the routed experts of the 128-expert decode batch (average 4 bits), on top of the shared expert's output
        _experts(64, 128, 2048, 768, 8, skew=1.0, padded=0.05, name="experts_decode"),
        # a 4096-token prompt through 64 experts
        _experts(4096, 64, 4096, 1408, 6, name="experts_prompt"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_route(rng):
    groups = rng.choice([1, 1, 1, 2, 4, 8])
    per = _log(rng, 4, 512 // groups if groups > 1 else 256)
    E = groups * per
    keep = rng.randint(1, groups)
    k = min(rng.choice([1, 2, 4, 6, 8, 8, 11, 16]), keep * per)
    T = _log(rng, 1, 16384)
    return _route(T, E, k, rng.choice(["softmax", "sigmoid"]), rng.choice(["f32", "f32", "bf16", "f16"]),
                  groups, keep, rng.choice(["max", "top2"]) if groups > 1 else "max", rng.random() < 0.6, rng.random() < 0.7,
                  rng.choice([1.0, 1.0, 2.5]), rng.choice([0.0, 0.0, 0.3]) if T >= 8 else 0.0, rng.choice([0.0, 0.0, 0.1]),
                  rng.choice([0, 0, 1, 8]))


def _draw_linear(rng):
    act = rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid", "swiglu", "swiglu"])
    size = (lambda lo, hi: _log(rng, lo, hi)) if rng.random() < 0.4 else (lambda lo, hi: max(1, (_log(rng, lo, hi) + 63) // 64) * 64)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    return _linear(_log(rng, 1, 8192), size(16, 8192), size(64, 8192), act, dtype, rng.choice([dtype, dtype, "f32"]),
                   rng.random() < 0.5, rng.random() < 0.5, rng.choice([0, 0, 0, 8, 3]))


def _draw_experts(rng):
    E = _log(rng, 4, 128)
    d, F = 128 * rng.randint(1, 16), 128 * rng.randint(1, 12)
    T = _log(rng, 1, 2048)
    return _experts(T, E, d, F, rng.randint(1, min(8, E)), rng.choice(["mixed", "mixed", "3", "4", "8"]),
                    rng.choice([0.0, 1.0]), rng.choice([0.0, 0.0, 0.2]) if T >= 8 else 0.0, rng.random() < 0.7)


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        c = rng.choice([_draw_route, _draw_linear, _draw_linear, _draw_experts])(rng)
        if _cost(c) <= top:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        live = T * (1.0 - c["padded"])   # the logits of padded tokens need not be read
        return {"bytes": live * E * BYTES[c["dtype"]] + T * k * 8 + E * 4 + (E * 4 if c["bias"] else 0) + (T if c["padded"] else 0),
                "flops": live * E * 10}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        R = 2 * N if c["act"] == "swiglu" else N
        return {"bytes": (M + R) * K * 2 + M * N * BYTES[c["out"]] * (2 if c["residual"] else 1) + (4 * R if c["bias"] else 0),
                "flops": 2 * M * R * K}
    T, E, d, F, k = c["T"], c["E"], c["d"], c["F"], c["k"]
    live = max(1.0, T * (1.0 - c["padded"]))
    p = _popularity(E, c["skew"])
    hit = sum(1.0 - (1.0 - min(1.0, k * q)) ** live for q in p)   # experts that some token takes
    bits = {"mixed": 4.0}.get(c["bits"]) or float(c["bits"])
    return {"bytes": hit * 3 * d * F * bits / 8 + T * d * 2 * (3 if c["residual"] else 2) + T * k * 8,
            "flops": 6 * d * F * live * k}


def _popularity(E, skew):
    p = [(e + 1) ** -skew for e in range(E)]
    return [q / sum(p) for q in p]


def _mixed_bits(E, bits):
    """Widths of the experts: one of them for all, or an average of four bits, wider for the more popular."""
    if bits != "mixed":
        return [int(bits)] * E
    return [8 if e % 8 == 0 else (4 if e % 8 in (1, 2, 3) else 3) for e in range(E)]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=gen, device=dev)  # noqa: E731
    c = dict(case)
    if c["op"] == "route":
        s = _inputs_route(c, randn, rand)
    elif c["op"] == "linear":
        s = _inputs_linear(c, randn)
    else:
        s = _inputs_experts(c, randn, rand)
    s["case"] = c
    if own:
        _own_handle(s)
    return s


def _inputs_route(c, randn, rand):
    T, E = c["T"], c["E"]
    buf = randn(T, E + c["pad_cols"]) * 1.5
    logits = buf.to(DTYPES[c["dtype"]])[:, :E]
    if c["absent"]:
        gone = rand(E) < c["absent"]
        gone[: max(1, E // 2)] = False
        logits.masked_fill_(gone, -math.inf)
    mask = rand(T) >= c["padded"] if c["padded"] else None
    bias = randn(E) * 0.1 if c["bias"] else None
    return dict(logits=logits, mask=mask, bias=bias)


def _inputs_linear(c, randn):
    M, N, K = c["M"], c["N"], c["K"]
    R = 2 * N if c["act"] == "swiglu" else N
    t = DTYPES[c["dtype"]]
    x = randn(M, K + c["pad"]).to(t)[:, :K]
    w = (randn(R, K + c["pad"]) * K ** -0.5).to(t)[:, :K]
    bias = randn(R) * 0.1 if c["bias"] else None
    residual = randn(M, N).to(DTYPES[c["out"]]) if c["residual"] else None
    return dict(x=x, w=w, bias=bias, residual=residual)


def _inputs_experts(c, randn, rand):
    T, E, d, F, k = c["T"], c["E"], c["d"], c["F"], c["k"]
    masters = [randn(E, F, d).mul_(0.02), randn(E, F, d).mul_(0.02), randn(E, d, F).mul_(0.02)]
    x = randn(T, d).to(torch.bfloat16)
    # the choice of a router whose popular experts are the first ones
    pop = torch.tensor(_popularity(E, c["skew"]), device=x.device).log()
    z = pop + 1.0 * -torch.log(-torch.log(rand(T, E).clamp_(1e-9, 1 - 1e-7)))
    top, ids = z.topk(k, dim=1)
    g = torch.softmax(top, dim=1)
    ids = ids.to(torch.int32)
    if c["padded"]:
        ids[rand(T) < c["padded"]] = -1
    residual = randn(T, d).to(torch.bfloat16) if c["residual"] else None
    s = dict(x=x, ids=ids, g=g, residual=residual, bits=_mixed_bits(E, c["bits"]))
    if own:
        s["masters"] = masters
    else:
        s["w1"], s["w3"], s["w2"] = _quantized(masters, s["bits"])
    return s


def _quantized(masters, bits):
    """The weights that the pages stand for, in fp32: round(w / s) s with one scale per expert, s = max|w| / (2^(b-1) - 1)."""
    qmax = torch.tensor([2 ** (b - 1) - 1 for b in bits], dtype=torch.float64, device=masters[0].device)
    top = torch.stack([m.abs().amax(dim=(1, 2)) for m in masters]).amax(dim=0)
    s = (top.double() / qmax).float().view(-1, 1, 1)
    return [m.div_(s).round_().mul_(s) for m in masters]


def _own_handle(s):
    from mixed_precision_weight_page_amd import PagedMoELayer
    c = s["case"]
    if c["op"] == "route":
        s["layer"] = PagedMoELayer(c["E"], 128, 128, c["k"], max_tokens=c["T"])
    elif c["op"] == "experts":
        layer = PagedMoELayer(c["E"], c["d"], c["F"], c["k"], max_tokens=c["T"])
        layer.bind_masters(*s["masters"])
        layer.alloc_pool(layer.pool_bytes_for_bits(s["bits"]))
        layer.alloc_workspace()
        layer.quantize_experts(s["bits"])
        s["layer"] = layer


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "linear": _own_linear, "experts": _own_experts}[op](state)
    return {"route": _plain_route, "linear": _plain_linear, "experts": _plain_experts}[op](state)


def _own_route(s):
    c = s["case"]
    ids, g, counts = s["layer"].route_gated(s["logits"], score=c["score"], bias=s["bias"], n_group=c["groups"],
                                            topk_group=c["keep"], group_score=c["group_score"], renorm=c["renorm"],
                                            scale=c["scale"], mask=s["mask"])
    return dict(ids=ids, g=g, counts=counts)


def _own_linear(s):
    from mixed_precision_weight_page_amd import linear
    c = s["case"]
    return linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"], out_dtype=DTYPES[c["out"]])


def _own_experts(s):
    return s["layer"].moe_forward_routed(s["x"], s["ids"], s["g"], residual=s["residual"], out_dtype=torch.bfloat16)


def _plain_route(s):
    # in 64 bits: a choice between two scores that are nearly equal must not hang on a rounding
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    raw = s["logits"]
    ok = raw > torch.finfo(raw.dtype).min
    if s["mask"] is not None:
        ok = ok & s["mask"][:, None]
    l = raw.double().masked_fill(~ok, -math.inf)
    if c["score"] == "softmax":
        m = l.amax(dim=1, keepdim=True)
        e = torch.exp(l - m.masked_fill(m == -math.inf, 0.0))
        p = e / e.sum(dim=1, keepdim=True).clamp_min(1e-300)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    choice = p + s["bias"].double() if s["bias"] is not None else p
    choice = choice.masked_fill(~ok, -math.inf)
    if G > 1:
        by = choice.view(T, G, E // G)
        if c["group_score"] == "top2":
            two = by.sort(dim=2, descending=True)[0][:, :, :2]
            # a group with one expert to be had counts that one, an empty one comes last
            score = two.masked_fill(two == -math.inf, 0.0).sum(dim=2).masked_fill(two[:, :, 0] == -math.inf, -math.inf)
        else:
            score = by.amax(dim=2)
        best = score.sort(dim=1, descending=True, stable=True)[1][:, : c["keep"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=raw.device).scatter_(1, best, True)
        choice = by.masked_fill(~kept[:, :, None], -math.inf).view(T, E)
    value, at = choice.sort(dim=1, descending=True, stable=True)
    value, at = value[:, :k], at[:, :k]
    took = value > -math.inf
    g = p.gather(1, at).masked_fill(~took, 0.0)
    if c["renorm"]:
        g = g / g.sum(dim=1, keepdim=True).clamp_min(1e-300)
    ids = at.masked_fill(~took, -1)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=raw.device)
    counts.index_add_(0, ids.masked_fill(~took, E).view(-1), torch.ones(T * k, dtype=torch.int32, device=raw.device))
    return dict(ids=ids.to(torch.int32), g=(g * c["scale"]).float(), counts=counts[:E])


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    return z


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"]
    if c["act"] == "swiglu":
        z = _act(z[:, : c["N"]], "silu") * z[:, c["N"]:]
    else:
        z = _act(z, c["act"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(DTYPES[c["out"]])


def _plain_experts(s):
    # the pairs of each expert side by side, every expert padded to the busiest one's count
    c = s["case"]
    T, E, d, k = c["T"], c["E"], c["d"], c["k"]
    flat = s["ids"].view(-1).long()
    key = flat.masked_fill(flat < 0, E)
    order = key.sort(stable=True)[1]
    count = torch.zeros(E + 1, dtype=torch.long, device=flat.device).index_add_(0, key, torch.ones_like(key))
    first = count.cumsum(0) - count
    place = torch.empty_like(key)
    place[order] = torch.arange(T * k, device=flat.device) - first[key[order]]
    room = max(1, int(count[:E].max()))
    live = flat >= 0
    row = (flat * room + place).masked_fill(~live, E * room)
    xs = torch.zeros((E * room + 1, d), dtype=torch.float32, device=flat.device)
    xs[row] = s["x"].float().repeat_interleave(k, dim=0)
    xs = xs[: E * room].view(E, room, d)
    a = torch.bmm(xs, s["w1"].transpose(1, 2))
    h = _act(a, "silu") * torch.bmm(xs, s["w3"].transpose(1, 2))
    o = torch.bmm(h, s["w2"].transpose(1, 2)).view(E * room, d)
    part = o[row.clamp_max(E * room - 1)].masked_fill(~live[:, None], 0.0)
    y = (part.view(T, k, d) * s["g"][:, :, None]).sum(dim=1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "linear": _exact_linear, "experts": _exact_experts}[case["op"]](s)


def _exact_route(s):
    """Weights of the chosen experts, each from its own logarithm; the choice by a mask taken away expert by expert."""
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    z = s["logits"].to(torch.float64)
    none = ~(s["logits"] > torch.finfo(s["logits"].dtype).min)
    if s["mask"] is not None:
        none = none | ~s["mask"].view(T, 1)
    z = torch.where(none, torch.full_like(z, -math.inf), z)
    if c["score"] == "softmax":
        logp = z - torch.logsumexp(z, dim=1, keepdim=True)
    else:
        logp = -torch.logaddexp(torch.zeros_like(z), -z)
    logp = torch.where(none, torch.full_like(z, -math.inf), logp)
    pick = torch.exp(logp)
    if s["bias"] is not None:
        pick = pick + s["bias"].to(torch.float64)
    pick = torch.where(none, torch.full_like(z, -math.inf), pick)
    index = torch.arange(E, device=z.device)
    low = torch.full((T, 1), -math.inf, dtype=torch.float64, device=z.device)
    if G > 1:
        score = []
        for q in range(G):
            part = pick[:, q * (E // G):(q + 1) * (E // G)]
            top = part.max(dim=1)[0]
            if c["group_score"] == "top2" and E // G > 1:
                second = part.topk(2, dim=1)[0][:, 1]
                top = top + torch.where(second == -math.inf, torch.zeros_like(second), second)
            score.append(top)
        score = torch.stack(score, dim=1)
        place = torch.arange(G, device=z.device)
        ahead = (score[:, None, :] > score[:, :, None]) | ((score[:, None, :] == score[:, :, None]) & (place[None, :] < place[:, None]))
        out = ahead.sum(dim=2) >= c["keep"]
        pick = torch.where(out.repeat_interleave(E // G, dim=1), torch.full_like(pick, -math.inf), pick)
    logs = []
    for _ in range(k):
        best = pick.max(dim=1, keepdim=True)[0]
        at = torch.where(pick == best, index, E).min(dim=1, keepdim=True)[0]
        logs.append(torch.where(best > -math.inf, logp.gather(1, at), low))
        pick = pick.scatter(1, at, -math.inf)
    logs = torch.cat(logs, dim=1)
    if c["renorm"]:
        total = torch.logsumexp(logs, dim=1, keepdim=True)
        logs = torch.where(logs > -math.inf, logs - total, logs)
    return dict(ids=None, g=torch.exp(logs) * c["scale"], counts=None)


def _exact_linear(s):
    c = s["case"]
    N = c["N"]
    w = s["w"].double()
    z = torch.matmul(w, s["x"].double().t()).t()
    if s["bias"] is not None:
        z = z + s["bias"].double()
    sig = lambda v: torch.exp(-torch.logaddexp(torch.zeros_like(v), -v))  # noqa: E731
    act = c["act"]
    if act == "swiglu":
        y = z[:, :N] * sig(z[:, :N]) * z[:, N:]
    elif act == "silu":
        y = z * sig(z)
    elif act == "sigmoid":
        y = sig(z)
    elif act == "relu":
        y = torch.where(z > 0, z, torch.zeros_like(z))
    elif act == "gelu":
        y = 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    elif act == "gelu_tanh":
        y = z * sig(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    else:
        y = z
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_experts(s):
    c = s["case"]
    x = s["x"].double()
    y = torch.zeros_like(x) if s["residual"] is None else s["residual"].double()
    for e in range(c["E"]):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        xe = x[t]
        a = xe @ s["w1"][e].double().t()
        h = a * torch.exp(-torch.logaddexp(torch.zeros_like(a), -a)) * (xe @ s["w3"][e].double().t())
        y.index_add_(0, t, (h @ s["w2"][e].double().t()) * s["g"][t, j].double()[:, None])
    return y
