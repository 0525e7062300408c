"""Operators in front of and beside the expert layer, as cases to measure and compare.

Four operators of a mixture-of-experts block whose dense weights are kept in 16 or in 8 bits:

* ``norm``      root-mean-square norm of the residual stream after an addition, in 16 bits or in e4m3 with scales
* ``quantize``  e4m3 values with a scale for each 128 columns of a row (activations) or each 128 x 128 tile (weights)
* ``linear8``   a dense product of such operands, with bias, activation and residual
* ``grouped``   products grouped by expert with ragged sizes, of 16-bit or e4m3 operands

Where ``own`` is false, ``run`` computes them in plain torch operations; where it is true, with the package's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
BLOCK = 128        # columns (and rows) of a scale
TOP = 448.0        # the largest value of e4m3
LEAST = 2.0 ** -100   # a block's largest magnitude counts as this at least


# ---------------------------------------------------------------- cases

def _norm(T, n, dtype="bf16", out="bf16", residual="", weight="bf16", pad=0, name=None):
    c = dict(op="norm", T=T, n=n, dtype=dtype, out=out, residual=residual, weight=weight, pad=pad)
    return dict(c, name=name) if name else c


def _quantize(E, M, K, dtype="bf16", tile=False, pad=0, name=None):
    c = dict(op="quantize", E=E, M=M, K=K, dtype=dtype, tile=tile, pad=pad)
    return dict(c, name=name) if name else c


def _linear8(M, N, K, act="none", out="bf16", bias=False, residual=False, pad=0, name=None):
    c = dict(op="linear8", M=M, N=N, K=K, act=act, out=out, bias=bias, residual=residual, pad=pad)
    return dict(c, name=name) if name else c


def _grouped(R, E, N, K, dtype="bf16", act="none", out="bf16", bias=False, residual=False, skew=0.0, behind=0, tokens=0, name=None):
    c = dict(op="grouped", R=R, E=E, N=N, K=K, dtype=dtype, act=act, out=out, bias=bias, residual=residual, skew=skew,
             behind=behind, tokens=tokens)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a single stream, on its way into an 8-bit product: launch latency
        _norm(1, 4096, out="e4m3", residual="bf16", name="norm_one_token"),
        # a batch of odd length and width in fp16, rows of a wider buffer, fp32 weights
        _norm(1003, 2051, "f16", "f16", weight="f32", pad=5, name="norm_ragged"),
        # a long prompt: the block's output joins the residual stream, the next product reads 8 bits
        _norm(16384, 4096, out="e4m3", residual="bf16", name="norm_prompt"),
        # SwiGLU rows of a 4096-token prompt's pairs (top-6, d_ff 1408) before the experts' down products
        _quantize(1, 24576, 1408, name="quantize_rows"),
        # a shared expert's gate and up weights from fp32 masters (d 4096, d_ff 14336), once per model
        _quantize(2, 14336, 4096, "f32", tile=True, name="quantize_weights"),
        # shared expert, 16 tokens: gate and up in one pass over the weights (d 4096, d_ff 14336)
        _linear8(16, 14336, 4096, "swiglu", name="linear8_shared_up_decode"),
        # odd sizes, rows of any alignment, everything in the epilogue
        _linear8(777, 1001, 700, "gelu", "f16", bias=True, residual=True, pad=5, name="linear8_odd"),
        # a square-ish dense layer over a long prompt
        _linear8(8192, 4096, 4096, "gelu_tanh", bias=True, residual=True, name="linear8_prompt"),
        # a decode batch's pairs (64 tokens, top-8) over 128 experts, popular ones first: gate and up, 16-bit weights
        _grouped(512, 128, 768, 2048, act="swiglu", skew=1.0, tokens=64, name="grouped_up_decode"),
        # the same batch's down products from 8-bit weights
        _grouped(512, 128, 2048, 768, "e4m3", skew=1.0, behind=24, name="grouped_down_decode8"),
        # a 4096-token prompt's pairs (top-6) through 64 experts: gate and up, each token's 8-bit row read where it lies
        _grouped(24576, 64, 1408, 4096, "e4m3", "swiglu", tokens=4096, name="grouped_up_prompt8"),
        # the same prompt's down products in 16 bits
        _grouped(24576, 64, 4096, 1408, skew=0.3, out="f32", name="grouped_down_prompt"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """Three of five whole multiples of 64, as a model's widths are; the others any."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.4 else max(64, (n + 63) // 64 * 64)


def _draw_norm(rng):
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    return _norm(_log(rng, 1, 16384), _width(rng, 1, 16384), dtype, rng.choice(["e4m3", dtype, "f32", "bf16"]),
                 rng.choice(["", dtype, "f32"]), rng.choice(["", dtype, "f32"]), rng.choice([0, 0, 8, 3]))


def _draw_quantize(rng):
    return _quantize(rng.choice([1, 1, 2, 8]), _log(rng, 1, 16384), _width(rng, 16, 14336), rng.choice(["bf16", "f16", "f32"]),
                     rng.random() < 0.5, rng.choice([0, 0, 3]))


ACTS = ["none", "none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid", "swiglu", "swiglu"]


def _draw_linear8(rng):
    return _linear8(_log(rng, 1, 8192), _width(rng, 16, 8192), _width(rng, 64, 8192), rng.choice(ACTS),
                    rng.choice(["bf16", "bf16", "f16", "f32"]), rng.random() < 0.5, rng.random() < 0.5, rng.choice([0, 0, 0, 16, 3]))


def _draw_grouped(rng):
    R = _log(rng, 1, 24576)
    dtype = rng.choice(["bf16", "f16", "e4m3", "e4m3"])
    return _grouped(R, _log(rng, 1, 128), _width(rng, 32, 4096), _width(rng, 64, 4096), dtype, rng.choice(ACTS),
                    rng.choice(["bf16", "f32"]), rng.random() < 0.3, rng.random() < 0.3, rng.choice([0.0, 0.5, 1.0]),
                    rng.choice([0, 0, 1, 37]), rng.choice([0, 0, (R + 3) // 4]))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        c = rng.choice([_draw_norm, _draw_quantize, _draw_linear8, _draw_linear8, _draw_grouped, _draw_grouped])(rng)
        if _cost(c) <= top and (c["op"] != "grouped" or c["E"] * c["N"] * c["K"] <= 4e8):
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    c = case
    if c["op"] == "norm":
        T, n = c["T"], c["n"]
        b = BYTES[c["dtype"]] + BYTES[c["out"]] + (2 * BYTES[c["residual"]] if c["residual"] else 0)
        scales = 4 * T * _blocks(n) if c["out"] == "e4m3" else 0
        return {"bytes": T * n * b + (n * BYTES[c["weight"]] if c["weight"] else 0) + scales, "flops": T * n * 8}
    if c["op"] == "quantize":
        E, M, K = c["E"], c["M"], c["K"]
        return {"bytes": E * (M * K * (BYTES[c["dtype"]] + 1) + 4 * (_blocks(M) if c["tile"] else M) * _blocks(K)), "flops": E * M * K * 4}
    if c["op"] == "linear8":
        M, N, K = c["M"], c["N"], c["K"]
        R = 2 * N if c["act"] == "swiglu" else N
        return {"bytes": (M + R) * K + 4 * (M + _blocks(R)) * _blocks(K) + M * N * BYTES[c["out"]] * (2 if c["residual"] else 1) +
                (4 * R if c["bias"] else 0), "flops": 2 * M * R * K}
    R, E, N, K = c["R"], c["E"], c["N"], c["K"]
    W = 2 * N if c["act"] == "swiglu" else N
    hit = sum(1.0 - (1.0 - q) ** R for q in _popularity(E, c["skew"]))   # experts with a row
    rows = c["tokens"] or R
    b = hit * W * K * BYTES[c["dtype"]] + rows * K * BYTES[c["dtype"]] + R * N * BYTES[c["out"]] * (2 if c["residual"] else 1)
    if c["dtype"] == "e4m3":
        b += 4 * _blocks(K) * (rows + hit * _blocks(W))
    return {"bytes": b + (4 * hit * W if c["bias"] else 0) + (4 * R if c["tokens"] else 0) + 4 * E, "flops": 2 * R * W * K}


def _popularity(E, skew):
    p = [(e + 1) ** -skew for e in range(E)]
    return [q / sum(p) for q in p]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    c = dict(case)
    s = {"norm": _inputs_norm, "quantize": _inputs_quantize, "linear8": _inputs_linear8}.get(c["op"])
    s = s(c, randn) if s else _inputs_grouped(c, randn, lambda *q: torch.rand(q, generator=gen, device=dev))
    s["case"] = c
    return s


def _stream_rows(rows, cols, randn):
    """Rows of a residual stream: some channels far larger than the others, rows of different size."""
    v = randn(rows, cols)
    v *= torch.where(randn(cols) > 2.2, 20.0, 1.0)
    return v.mul_(torch.exp(0.5 * randn(rows, 1)))


def _padded(v, pad, dtype):
    """v as a view of a buffer whose rows are `pad` elements longer."""
    if not pad:
        return v.to(dtype)
    wide = torch.zeros((*v.shape[:-1], v.shape[-1] + pad), dtype=dtype, device=v.device)
    wide[..., : v.shape[-1]] = v.to(dtype)
    return wide[..., : v.shape[-1]]


def _inputs_norm(c, randn):
    T, n = c["T"], c["n"]
    x = _padded(_stream_rows(T, n, randn), c["pad"], DTYPES[c["dtype"]])
    residual = _stream_rows(T, n, randn).to(DTYPES[c["residual"]]) if c["residual"] else None
    weight = (1.0 + 0.2 * randn(n)).to(DTYPES[c["weight"]]) if c["weight"] else None
    return dict(x=x, residual=residual, weight=weight)


def _inputs_quantize(c, randn):
    E, M, K = c["E"], c["M"], c["K"]
    v = randn(E, M, K).mul_(K ** -0.5) if c["tile"] else _stream_rows(E * M, K, randn).view(E, M, K)
    v = _padded(v, c["pad"], DTYPES[c["dtype"]])
    return dict(x=v[0] if E == 1 else v)


def _eight(v, tile, pad=0):
    """e4m3 values of v [..., M, K] and their scales, as a user of 8-bit products has them: rows' scales lie block by block."""
    q, s = _quantized(v, tile)
    if not tile:
        s = s.transpose(-1, -2).contiguous().transpose(-1, -2)
    return _padded(q, pad, torch.float8_e4m3fn), s


def _inputs_linear8(c, randn):
    M, N, K = c["M"], c["N"], c["K"]
    x = _eight(_stream_rows(M, K, randn), False, c["pad"])
    halves = 2 if c["act"] == "swiglu" else 1   # the gate and the up rows have tiles of their own
    w, ws = _eight(randn(halves, N, K).mul_(K ** -0.5), True)
    bias = randn(halves * N) * 0.1 if c["bias"] else None
    residual = randn(M, N).to(DTYPES[c["out"]]) if c["residual"] else None
    return dict(x=x, w=(_padded(w.view(halves * N, K), c["pad"], w.dtype), ws.view(-1, ws.shape[-1])), bias=bias, residual=residual)


def _inputs_grouped(c, randn, rand):
    R, E, N, K = c["R"], c["E"], c["N"], c["K"]
    halves = 2 if c["act"] == "swiglu" else 1
    rows = c["tokens"] or R + c["behind"]
    # rows of each expert, drawn by its popularity
    edge = torch.tensor(_popularity(E, c["skew"]), device="cuda").cumsum(0)
    expert = torch.searchsorted(edge, rand(R)).clamp_max(E - 1)
    count = torch.zeros(E, dtype=torch.int64, device="cuda").index_add_(0, expert, torch.ones_like(expert))
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = count.cumsum(0)
    x = _stream_rows(rows, K, randn)
    w = randn(E * halves, N, K).mul_(K ** -0.5)
    if c["dtype"] == "e4m3":
        x = _eight(x, False)
        w, ws = _eight(w, True)
        w = (w.view(E, halves * N, K), ws.view(E, -1, ws.shape[-1]))
    else:
        x, w = x.to(DTYPES[c["dtype"]]), w.to(DTYPES[c["dtype"]]).view(E, halves * N, K)
    bias = randn(E, halves * N) * 0.1 if c["bias"] else None
    place = None
    if c["tokens"]:
        place = torch.zeros(R + c["behind"], dtype=torch.int32, device="cuda")
        place[:R] = (rand(R) * c["tokens"]).to(torch.int32).clamp_max(c["tokens"] - 1)
    # rows behind the last expert's stay as they are
    y = torch.full((R + c["behind"], N), 0.5, dtype=DTYPES[c["out"]], device="cuda")
    residual = randn(R + c["behind"], N).to(DTYPES[c["out"]]) if c["residual"] else None
    return dict(x=x, w=w, bias=bias, offsets=offsets, rows=place, y=y, residual=residual)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "quantize": _own_quantize, "linear8": _own_linear8, "grouped": _own_grouped}[op](state)
    return {"norm": _plain_norm, "quantize": _plain_quantize, "linear8": _plain_linear8, "grouped": _plain_grouped}[op](state)


def _own_norm(s):
    from mixed_precision_weight_page_amd import rms_norm
    c = s["case"]
    y = rms_norm(s["x"], s["weight"], 1e-6, residual=s["residual"], out_dtype=DTYPES[c["out"]])
    y, h = y if s["residual"] is not None else (y, None)
    out = dict(q=y[0], scale=y[1]) if c["out"] == "e4m3" else dict(y=y)
    return out if h is None else dict(out, h=h)


def _own_quantize(s):
    from mixed_precision_weight_page_amd import quantize_fp8
    q, scale = quantize_fp8(s["x"], block="tile" if s["case"]["tile"] else "row")
    return dict(q=q, scale=scale)


def _own_linear8(s):
    from mixed_precision_weight_page_amd import linear_fp8
    c = s["case"]
    return linear_fp8(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"], out_dtype=DTYPES[c["out"]])


def _own_grouped(s):
    from mixed_precision_weight_page_amd import grouped_linear
    return grouped_linear(s["x"], s["offsets"], s["w"], bias=s["bias"], act=s["case"]["act"], residual=s["residual"], rows=s["rows"], y=s["y"])


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = (h + s["residual"].float()).to(s["residual"].dtype)
    written, h = h, h.float()
    r = 1.0 / torch.sqrt(h.double().square().mean(dim=1, keepdim=True) + 1e-6)
    z = h * s["weight"].float() if s["weight"] is not None else h
    if c["out"] == "e4m3":
        q, m = _codes(z, False)
        out = dict(q=q, scale=(m * r / TOP).float())
    else:
        out = dict(y=(z * r.float()).to(DTYPES[c["out"]]))
    return out if s["residual"] is None else dict(out, h=written)


def _codes(v, tile):
    """e4m3 values 448 v / m and m, in 64 bits: m the largest magnitude of each block of v [..., M, K]."""
    M, K = v.shape[-2:]
    down = BLOCK if tile else 1
    full = torch.zeros((*v.shape[:-2], (M + down - 1) // down * down, _blocks(K) * BLOCK), dtype=torch.float32, device=v.device)
    full[..., :M, :K] = v.float()
    cut = full.view(*v.shape[:-2], -1, down, _blocks(K), BLOCK)
    m = cut.abs().nan_to_num(0.0, math.inf).amax(dim=(-3, -1), keepdim=True).clamp_min(LEAST).double()
    # two values may be as far from one code as from the next: 64 bits say which are
    q = (cut.double() * TOP / m).float().view(full.shape)[..., :M, :K]
    return q.to(torch.float8_e4m3fn), m[..., 0, :, 0]


def _quantized(v, tile):
    q, m = _codes(v, tile)
    return q, (m / TOP).float()


def _plain_quantize(s):
    q, scale = _quantized(s["x"], s["case"]["tile"])
    return dict(q=q, scale=scale)


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


def _finish(z, c, bias, residual):
    if bias is not None:
        z = z + bias
    if c["act"] == "swiglu":
        z = _act(z[..., : c["N"]], "silu") * z[..., c["N"]:]
    else:
        z = _act(z, c["act"])
    return z if residual is None else z + residual.float()


def _values(q, scale):
    """What rows' e4m3 values and scales stand for, in 32 bits."""
    return q.float() * scale.repeat_interleave(BLOCK, dim=-1)[..., : q.shape[-1]]


def _weights(q, scale, halves):
    """What tiles' e4m3 values and scales stand for: [..., halves, N, K] with the tiles of each half from its first row."""
    *lead, R, K = q.shape
    cut = q.float().view(*lead, halves, R // halves, K)
    s = scale.view(*lead, halves, -1, scale.shape[-1])
    s = s.repeat_interleave(BLOCK, dim=-2)[..., : R // halves, :].repeat_interleave(BLOCK, dim=-1)[..., :K]
    return (cut * s).view(*lead, R, K)


def _plain_linear8(s):
    c = s["case"]
    w = _weights(s["w"][0].contiguous(), s["w"][1], 2 if c["act"] == "swiglu" else 1)
    return _finish(_values(*s["x"]) @ w.t(), c, s["bias"], s["residual"]).to(DTYPES[c["out"]])


def _plain_grouped(s):
    # every expert's rows side by side, padded to the busiest one's count
    c = s["case"]
    R, E = c["R"], c["E"]
    if c["dtype"] == "e4m3":
        x, w = _values(*s["x"]), _weights(*s["w"], 2 if c["act"] == "swiglu" else 1)
    else:
        x, w = s["x"].float(), s["w"].float()
    first = s["offsets"].long()
    at = torch.arange(R, device=x.device)
    expert = torch.searchsorted(first, at, right=True) - 1
    room = max(1, int((first[1:] - first[:-1]).max()))
    row = expert * room + at - first[expert]
    xs = torch.zeros((E * room, x.shape[1]), dtype=torch.float32, device=x.device)
    xs[row] = x[s["rows"][:R].long()] if s["rows"] is not None else x[:R]
    z = torch.bmm(xs.view(E, room, -1), w.transpose(1, 2)).view(E * room, -1)[row]
    bias = s["bias"][expert] if s["bias"] is not None else None
    residual = s["residual"][:R] if s["residual"] is not None else None
    y = s["y"]
    y[:R] = _finish(z, c, bias, residual).to(y.dtype)
    return y


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "quantize": _exact_quantize, "linear8": _exact_linear8, "grouped": _exact_grouped}[case["op"]](s)


def _spread(v, cols):
    """One value for each column from one for each 128."""
    return v[..., torch.arange(cols, device=v.device) // BLOCK]


def _exact_norm(s):
    c = s["case"]
    h = s["x"].to(torch.float64)
    out = {}
    if s["residual"] is not None:
        h = h + s["residual"].to(torch.float64)
        out["h"] = h
        h = h.to(s["residual"].dtype).to(torch.float64)   # what is normalised is what is written
    size = torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / c["n"] + 1e-6)
    y = h / size if s["weight"] is None else h / size * s["weight"].to(torch.float64)
    if c["out"] != "e4m3":
        return dict(out, y=y)
    m = torch.stack([part.abs().amax(dim=1) for part in y.split(BLOCK, dim=1)], dim=1)
    m = torch.maximum(m, LEAST / size)
    return dict(out, q=y / _spread(m, c["n"]) * TOP, scale=m / TOP)


def _exact_quantize(s):
    c = s["case"]
    v = s["x"].to(torch.float64)
    size = torch.stack([part.abs().amax(dim=-1) for part in v.split(BLOCK, dim=-1)], dim=-1)   # [..., M, blocks]
    if c["tile"]:
        m = torch.stack([part.amax(dim=-2) for part in size.split(BLOCK, dim=-2)], dim=-2).clamp_min(LEAST)
        wide = m[..., torch.arange(c["M"], device=v.device) // BLOCK, :]
    else:
        m = wide = size.clamp_min(LEAST)
    return dict(q=v / _spread(wide, c["K"]) * TOP, scale=m / TOP)


def _exact_finish(z, c, bias, residual):
    if bias is not None:
        z = z + bias.double()
    sig = lambda v: torch.exp(-torch.logaddexp(torch.zeros_like(v), -v))  # noqa: E731
    act, N = c["act"], c["N"]
    if act == "swiglu":
        z = z[:, :N] * sig(z[:, :N]) * z[:, N:]
    elif act == "silu":
        z = z * sig(z)
    elif act == "sigmoid":
        z = sig(z)
    elif act == "relu":
        z = torch.where(z > 0, z, torch.zeros_like(z))
    elif act == "gelu":
        z = 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    elif act == "gelu_tanh":
        z = z * sig(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z if residual is None else z + residual.double()


def _exact_product(x, w, halves):
    """x w^T block by block of K where the operands are (values, scales), else as it stands."""
    if not isinstance(w, tuple):
        return torch.matmul(w.double(), x.double().t()).t()
    (q, s), (v, t) = x, w
    N = v.shape[0] // halves
    z = torch.zeros((q.shape[0], v.shape[0]), dtype=torch.float64, device=q.device)
    tile = torch.arange(N, device=q.device) // BLOCK
    if halves == 2:
        tile = torch.cat([tile, tile + _blocks(N)])
    for b in range(_blocks(q.shape[1])):
        cols = slice(b * BLOCK, (b + 1) * BLOCK)
        z += q[:, cols].double() @ v[:, cols].double().t() * s[:, b, None].double() * t[tile, b].double()
    return z


def _exact_linear8(s):
    c = s["case"]
    return _exact_finish(_exact_product(s["x"], s["w"], 2 if c["act"] == "swiglu" else 1), c, s["bias"], s["residual"])


def _exact_grouped(s):
    c = s["case"]
    eight = c["dtype"] == "e4m3"
    y = s["y"].double()
    first = s["offsets"].tolist()
    for e in range(c["E"]):
        a, b = first[e], first[e + 1]
        if a == b:
            continue
        at = s["rows"][a:b].long() if s["rows"] is not None else torch.arange(a, b, device=y.device)
        x = tuple(v[at] for v in s["x"]) if eight else s["x"][at]
        w = tuple(v[e] for v in s["w"]) if eight else s["w"][e]
        y[a:b] = _exact_finish(_exact_product(x, w, 2 if c["act"] == "swiglu" else 1), c,
                               s["bias"][e] if s["bias"] is not None else None, s["residual"][a:b] if s["residual"] is not None else None)
    return y
