"""GPU tests of pw_linear against the product in float64.

Tolerance of an output, from arithmetic: the K products are exact in fp32
and summed in fp32 in some order, each sum off by at most one unit in the
last place (2^-23) of a partial sum of magnitude at most S = sum |x w| +
|bias|, so z is off by at most dz = (K + 2) 2^-23 S. The activations used
have slopes of at most 1.13, and their native exponential, reciprocal and
products add at most 2^-20 of |z| (SwiGLU: the product rule). The residual's
addition and the rounding to y's type add half a step each."""
import math

import pytest
import torch

from layer_cases import log

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def act64(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "sigmoid":
        return torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z * math.sqrt(0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def reference(x, w, bias, act, residual):
    """(y, bound before the last rounding) in float64 on the CPU."""
    x, w = x.double(), w.double()
    K = x.shape[1]
    z, S = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, S = z + bias.double(), S + bias.double().abs()
    dz = (K + 2) * 2.0 ** -23 * S
    if act == "swiglu":
        n = w.shape[0] // 2
        s = act64(z[:, :n], "silu")
        y = s * z[:, n:]
        ds = 1.13 * dz[:, :n] + 2.0 ** -20 * z[:, :n].abs()
        tol = ds * (z[:, n:].abs() + dz[:, n:]) + s.abs() * dz[:, n:] + 2.0 ** -23 * y.abs()
    else:
        y = act64(z, act)
        tol = 1.13 * dz + (2.0 ** -20 * z.abs().clamp_min(y.abs()) if act not in ("none", "relu") else 0.0)
    if residual is not None:
        y = y + residual.double()
        tol = tol + 2.0 ** -24 * (y.abs() + tol)
    return y, tol


def strided(rows, cols, pad, dtype, gen, scale=1.0):
    """A [rows, cols] view of a wider buffer whose other columns are NaN."""
    v = (torch.randn(rows, cols, generator=gen) * scale).to(dtype)
    buf = torch.full((rows, cols + pad), float("nan"), dtype=dtype)
    buf[:, :cols] = v
    return v, buf.cuda()[:, :cols]


def run(M, N, K, act="none", dtype="bf16", out="bf16", bias=False, residual=False, pads=(0, 0, 0, 0), alias=False, seed=0):
    from mixed_precision_weight_page_amd import linear
    gen = torch.Generator().manual_seed(seed + 131 * M + 17 * N + K)
    R = 2 * N if act == "swiglu" else N
    x, xd = strided(M, K, pads[0], DT[dtype], gen)
    w, wd = strided(R, K, pads[1], DT[dtype], gen, max(K, 1) ** -0.5)
    b = torch.randn(R, generator=gen) if bias else None
    r, rd = strided(M, N, pads[2], DT[out], gen) if residual else (None, None)
    log(f"linear {M}x{N}x{K} {act} {dtype}->{out} pads {pads}")
    guard = 3
    if alias:
        y = rd
    else:
        # y inside a larger buffer: what is around it stays
        buf = torch.full((M + 2, N + pads[3] + guard), 7.0, dtype=DT[out], device="cuda")
        y = buf[1:M + 1, :N]
    got = linear(xd, wd, None if b is None else b.cuda(), act, rd, y, DT[out])
    torch.cuda.synchronize()
    assert got.data_ptr() == y.data_ptr()
    ref, tol = reference(x, w, b, act, r)
    tol = tol + torch.finfo(DT[out]).eps / 2 * (ref.abs() + tol) + torch.finfo(DT[out]).tiny
    err = (y.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), float(err.max()))
    if not alias:
        whole = buf.cpu()
        whole[1:M + 1, :N] = 7.0
        assert bool((whole == 7.0).all()), "written outside y"
    return y


ACTS = ["none", "relu", "silu", "sigmoid", "gelu", "gelu_tanh", "swiglu"]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 16, 40, 70, 300])
def test_activations(act, M):
    run(M, 96, 136, act, bias=True, residual=True)
    run(M, 50, 72, act, "f16", "f32", bias=True)


SIZES = [(1, 1, 1), (1, 1, 0), (2, 3, 7), (15, 16, 8), (16, 17, 63), (17, 100, 64), (33, 260, 65), (48, 5, 520), (64, 64, 1000),
         (64, 9000, 40), (20, 8300, 129), (65, 1, 9), (65, 130, 64), (100, 33, 0), (127, 129, 200), (128, 128, 128), (130, 257, 72),
         (257, 64, 333), (513, 300, 24)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_sizes(M, N, K, act):
    run(M, N, K, act, "bf16", "f32", bias=True)
    run(M, N, K, act, "f16", "f16", residual=True)


# row distances: 16-byte rows, rows of other alignments, wide residual and y
@pytest.mark.parametrize("pads", [(8, 16, 4, 8), (1, 3, 5, 7), (0, 4, 0, 1), (2, 0, 1, 0)])
@pytest.mark.parametrize("M", [5, 64, 90, 600])
def test_strides(pads, M):
    run(M, 100, 96, "swiglu", bias=True, residual=True, pads=pads)
    run(M, 101, 83, "gelu", "f16", "f32", bias=True, residual=True, pads=pads)


# the tiles of large products: 256 x 256 and 128 x 128, ragged in every size
@pytest.mark.parametrize("M,N,K,act", [(2100, 2900, 200, "none"), (2049, 1500, 136, "swiglu"), (1000, 2000, 328, "silu"),
                                       (1025, 1100, 64, "swiglu"), (4100, 2050, 8, "none")])
def test_large_tiles(M, N, K, act):
    run(M, N, K, act, bias=True, residual=True)


# enough tiles of 192 x 256 for the phased kernel: every number of stages of
# 64 K values up to its slots and past them, whole and ragged
@pytest.mark.parametrize("K", [0, 8, 32, 40, 64, 96, 128, 136, 168, 520])
def test_phased_stages(K):
    run(4100, 2050, K, "none", bias=True)
    run(2305, 1990, K, "swiglu", "f16", "f16", residual=True)


# a size for each of the five tiles (64 x 64, 128 x 128, 128 rows x 256
# tokens, 192 x 256, 256 x 256), ragged, with fewer and more steps of K than
# its LDS holds
TILES = [(200, 300), (1100, 2300), (2100, 2900), (4000, 2800), (4000, 3900)]


@pytest.mark.parametrize("K", [0, 8, 64, 72, 200, 392])
@pytest.mark.parametrize("M,N", TILES)
def test_every_tile(M, N, K):
    run(M, N, K, "none", "bf16", "bf16", bias=True, residual=True)
    run(M, N // 2, K, "swiglu", "f16", "f32", residual=True, pads=(8, 16, 4, 4))


@pytest.mark.parametrize("M,N,K", [(16, 512, 8192), (1, 256, 14336), (512, 256, 8192)])
def test_long_sums(M, N, K):
    run(M, N, K, "none", "bf16", "f32")
    run(M, N, K, "swiglu", "bf16", "bf16", residual=True)


@pytest.mark.parametrize("M", [3, 64, 200, 700])
def test_residual_is_the_output(M):
    run(M, 160, 128, "none", residual=True, alias=True)
    run(M, 61, 70, "silu", "bf16", "f32", residual=True, alias=True, pads=(0, 0, 2, 2))


def test_offsets_past_32_bits():
    """x, y and residual with rows so far apart that the last ones lie more
    than 2^32 bytes on."""
    from mixed_precision_weight_page_amd import linear
    M, N, K, ld = 1100, 24, 40, (1 << 21) + 8
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(M, K, generator=gen).bfloat16()
    w = torch.randn(N, K, generator=gen).bfloat16()
    r = torch.randn(M, N, generator=gen).bfloat16()
    buf = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda").view(M, ld)
    buf[:, :K] = x.cuda()
    buf[:, 64:64 + N] = r.cuda()
    y = buf[:, 128:128 + N]
    linear(buf[:, :K], w.cuda(), residual=buf[:, 64:64 + N], y=y)
    linear(buf[:3, :K], w.cuda(), residual=buf[:3, 64:64 + N], y=buf[:3, 160:160 + N])
    ref, tol = reference(x, w, None, "none", r)
    tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert bool(((y.cpu().double() - ref).abs() <= tol).all())
    assert bool(((buf[:3, 160:160 + N].cpu().double() - ref[:3]).abs() <= tol[:3]).all())


def test_infinities_and_nans_stay_in_their_rows():
    from mixed_precision_weight_page_amd import linear
    for M in (20, 200):
        x = torch.randn(M, 128).bfloat16()
        w = torch.randn(64, 128).bfloat16().abs()
        x[3, 5], x[7, 0] = math.inf, math.nan
        x[3, :5], x[3, 6:] = 1.0, 1.0
        y = linear(x.cuda(), w.cuda()).cpu()
        assert bool((y[3] == math.inf).all()) and bool(y[7].isnan().all())
        rest = [i for i in range(M) if i not in (3, 7)]
        assert bool(y[rest].isfinite().all())


@pytest.mark.parametrize("M", [8, 400])
def test_captured_linear_replays(M):
    from mixed_precision_weight_page_amd import linear
    w = torch.randn(256, 192, device="cuda").bfloat16()
    x = torch.randn(M, 192, device="cuda").bfloat16()
    linear(x, w, act="swiglu")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = linear(x, w, act="swiglu")
    for i in range(3):
        x.copy_(torch.randn(M, 192, device="cuda"))
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, linear(x, w, act="swiglu"))


def test_another_stream():
    from mixed_precision_weight_page_amd import linear
    x, w = torch.randn(1000, 512).bfloat16(), torch.randn(256, 512).bfloat16()
    side = torch.cuda.Stream()
    xd, wd = x.cuda(), w.cuda()
    want = linear(xd, wd)
    torch.cuda.synchronize()
    y = linear(xd, wd, stream=side)
    del xd, wd
    junk = [torch.full((1000, 512), 9.0, device="cuda") for _ in range(4)]
    side.synchronize()
    assert torch.equal(y, want)
    del junk
