"""GPU tests of fp32 results of e4m3 operands (pw_linear_fp8,
pw_grouped_linear and moe_experts), where nothing of a product may be lost.

Whole numbers: codes are odd numbers up to 15 and, one in eight, multiples of
16 up to 240, and scales 1/2 or 1. Then every product and every sum over part
of K, in any order, is a multiple of 1/4 of magnitude below 2^22 (asserted), so
fp32 holds all of them and y has no rounding to make: it has to be equal. A
large product beside a small one is up to 2^16, so an instruction that drops
what is below 2^-13 of the largest would drop units.

Random codes: product_cases.reference's bound for exact products, fp32 sums."""
import pytest
import torch

from layer_cases import log
from product_cases import E4M3, eight_bits, reference, strided, tile_values, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def whole_codes(shape, gen):
    v = 2.0 * torch.randint(0, 8, shape, generator=gen) + 1.0
    large = torch.rand(shape, generator=gen) < 0.125
    v = torch.where(large, 16.0 * torch.randint(8, 16, shape, generator=gen), v)
    return torch.where(torch.rand(shape, generator=gen) < 0.5, -v, v)


def whole_scales(shape, gen):
    return 2.0 ** -torch.randint(0, 2, shape, generator=gen).float()


def exact(x, w):
    """x w^T in float64, both [rows, K]; every sum of parts of it fits fp32."""
    assert float((x.abs() @ w.abs().t()).max()) < 2.0 ** 22
    return x @ w.t()


# streamed weights, tiles of all sizes, rows of any alignment (pads)
DENSE = [(1, 300, 4096), (7, 130, 1168), (16, 4100, 512), (33, 700, 2048), (64, 4096, 1024), (128, 4096, 1024), (300, 260, 1168),
         (1000, 2048, 384), (2100, 2900, 272), (4100, 4000, 144), (7239, 1800, 400)]


@pytest.mark.parametrize("M,N,K", DENSE)
def test_dense_whole_numbers(M, N, K):
    from mixed_precision_weight_page_amd import linear_fp8
    gen = torch.Generator().manual_seed(M)
    x, w = whole_codes((M, K), gen), whole_codes((N, K), gen)
    xs, ws = whole_scales((M, -(-K // 128)), gen), whole_scales((-(-N // 128), -(-K // 128)), gen)
    want = exact(values(x, xs), tile_values(w, ws))
    log(f"whole numbers {M}x{N}x{K}")
    y = linear_fp8((x.to(E4M3).cuda(), xs.cuda()), (w.to(E4M3).cuda(), ws.cuda()), out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), want)


@pytest.mark.parametrize("pads", [(1, 3), (2, 1), (3, 5), (8, 8)])
@pytest.mark.parametrize("M,N,K", [(5, 300, 1167), (44, 60, 700), (90, 600, 1165), (1700, 1900, 261)])
def test_dense_whole_numbers_of_any_alignment(M, N, K, pads):
    from mixed_precision_weight_page_amd import linear_fp8
    gen = torch.Generator().manual_seed(M + pads[0])
    x, w = whole_codes((M, K), gen), whole_codes((N, K), gen)
    xs, ws = whole_scales((M, -(-K // 128)), gen), whole_scales((-(-N // 128), -(-K // 128)), gen)
    want = exact(values(x, xs), tile_values(w, ws))
    log(f"whole numbers {M}x{N}x{K} pads {pads}")
    y = linear_fp8((strided(x.to(E4M3), pads[0]), xs.cuda()), (strided(w.to(E4M3), pads[1]), ws.cuda()), out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), want)


COUNTS = [[1, 0, 2], [9] * 40, [4] * 128, [20, 0, 30, 17], [40, 100, 0, 7], [130, 257, 0, 1, 64], [700, 3, 900], [1100, 1300], [2500, 1800]]


@pytest.mark.parametrize("counts", COUNTS, ids=[f"{len(c)}e{sum(c)}r" for c in COUNTS])
@pytest.mark.parametrize("N,K,pads", [(260, 1168, (0, 0)), (1300, 272, (16, 0)), (70, 261, (2, 3)), (1300, 261, (1, 1))])
def test_grouped_whole_numbers(counts, N, K, pads):
    from mixed_precision_weight_page_amd import grouped_linear
    E, R = len(counts), sum(counts)
    gen = torch.Generator().manual_seed(R)
    first = [0, *torch.tensor(counts).cumsum(0).tolist()]
    tokens = R // 2 + 1
    rows = torch.randint(0, tokens, (R,), generator=gen)
    x, xs = whole_codes((tokens, K), gen), whole_scales((tokens, -(-K // 128)), gen)
    w, ws = whole_codes((E, N, K), gen), whole_scales((E, -(-N // 128), -(-K // 128)), gen)
    log(f"whole numbers {counts[:4]} {N}x{K} pads {pads}")
    y = grouped_linear((strided(x.to(E4M3), pads[0]), xs.cuda()), torch.tensor(first, dtype=torch.int32).cuda(),
                       (strided(w.to(E4M3), pads[1]), ws.cuda()), rows=rows.to(torch.int32).cuda(), out_dtype=torch.float32).cpu()
    x64 = values(x, xs)
    for e in range(E):
        p, q = first[e], first[e + 1]
        if p < q:
            assert torch.equal(y[p:q].double(), exact(x64[rows[p:q]], tile_values(w[e], ws[e]))), e


@pytest.mark.parametrize("M", [3, 40, 300, 1500])
@pytest.mark.parametrize("act,pads", [("none", (0, 0)), ("swiglu", (16, 0)), ("gelu", (1, 2)), ("swiglu", (3, 0))])
def test_random_codes(M, act, pads):
    """One octet of K to a few blocks, in which exact sums are close: rows whose channels differ by twenty times."""
    from mixed_precision_weight_page_amd import linear_fp8
    for N, K in ((200, 8), (70, 16), (300, 144), (900, 528)):
        gen = torch.Generator().manual_seed(M + K)
        halves = 2 if act == "swiglu" else 1
        x, xd = eight_bits((M, K), gen, False, pad=pads[0])
        w, wd = eight_bits((halves * N, K), gen, True, K ** -0.5, pads[1], halves)
        bias = torch.randn(halves * N, generator=gen)
        r = torch.randn(M, N, generator=gen)
        log(f"random codes {M}x{N}x{K} {act} pads {pads}")
        y = linear_fp8(xd, wd, bias.cuda(), act, r.cuda())
        assert y.dtype == torch.float32
        want, tol = reference(x, w, bias, act, r, torch.float32)
        assert bool(((y.cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("T", [1, 40, 600])
def test_experts_with_an_fp32_result(T):
    """The down products that moe_experts joins, from the codes of the SwiGLU rows that its first half leaves."""
    from mixed_precision_weight_page_amd import group_routes, grouped_linear, moe_experts, quantize_fp8
    E, k, d, F = 8, 3, 96, 16
    gen = torch.Generator().manual_seed(T)
    x = torch.randn(T, d, generator=gen).bfloat16().cuda()
    up = quantize_fp8((torch.randn(2 * E, F, d, generator=gen) * d ** -0.5).cuda(), "tile")
    up = type(up)(up.q.view(E, 2 * F, d), up.scale.view(E, -1, up.scale.shape[-1]))
    down = quantize_fp8((torch.randn(E, d, F, generator=gen) * F ** -0.5).cuda(), "tile")
    ids = torch.randint(-1, E, (T, k), generator=gen).to(torch.int32)
    g = torch.rand(T, k, generator=gen)
    residual = torch.randn(T, d, generator=gen)
    log(f"moe_experts {T} tokens, fp32")
    y = moe_experts(x, ids.cuda(), g.cuda(), up, down, residual.cuda()).cpu().double()
    offsets, rows, place = group_routes(ids.cuda(), E)
    h = quantize_fp8(grouped_linear(quantize_fp8(x), offsets, up, act="swiglu", rows=rows, out_dtype=torch.bfloat16))
    hv, place = values(h.q.float().cpu(), h.scale.cpu()), place.cpu()
    want, size, tol = residual.double(), residual.double().abs(), torch.zeros(T, d, dtype=torch.float64)
    for e in range(E):
        we = tile_values(down.q[e].float().cpu(), down.scale[e].cpu())
        for t, j in (ids == e).nonzero().tolist():
            o, ot = reference(hv[place[t, j]][None], we, None, "none", None, torch.float32)
            w = float(g[t, j])
            want[t] += w * o[0]
            size[t] += w * o[0].abs()
            tol[t] += w * ot[0]
    # k products and sums, each off by half a step of a sum of at most `size`
    tol = tol + (k + 1) * 2.0 ** -23 * (size + tol)
    assert bool(((y - want).abs() <= tol).all()), float(((y - want).abs() / tol).max())


@pytest.mark.parametrize("M,N,pad", [(254, 1, 0), (254, 1, 3), (254, 300, 0), (254, 5000, 0), (2540, 3000, 0), (2540, 3000, 1)])
def test_every_code_by_one(M, N, pad):
    """K = 1: y is the code's own value, for each of the finite ones."""
    from mixed_precision_weight_page_amd import linear_fp8
    codes = torch.arange(256, dtype=torch.uint8).view(E4M3)
    fine = codes[(torch.arange(256) & 127) != 127]
    x = fine.view(torch.uint8).repeat(M // 254)[:, None].view(E4M3)
    w = torch.ones(N, 1).to(E4M3)
    one = torch.ones((), device="cuda")
    for K in (1, 16):   # the others are zeros
        xk, wk = torch.zeros(M, K).to(E4M3), torch.zeros(N, K).to(E4M3)
        xk[:, :1], wk[:, :1] = x, w
        y = linear_fp8((strided(xk, pad), one.expand(M, 1)), (strided(wk, pad), one.expand(-(-N // 128), 1)), out_dtype=torch.float32)
        assert torch.equal(y.cpu(), x.float().expand(M, N))


@pytest.mark.parametrize("M", [5, 60, 200, 3000])
@pytest.mark.parametrize("pad", [0, 3])
def test_infinities_and_nans_stay_in_their_rows(M, pad):
    from mixed_precision_weight_page_amd import grouped_linear, linear_fp8
    gen = torch.Generator().manual_seed(M)
    for N in (130, 2000):
        x, (xq, xs) = eight_bits((M, 272), gen, False)
        w, (wq, ws) = eight_bits((N, 272), gen, True, pad=pad)
        xq, xs = xq.float().cpu(), xs.cpu().clone()
        xq[2, 0], xs[3, 1], xs[4, 0] = float("nan"), float("inf"), float("nan")
        xd = (strided(xq.to(E4M3), pad), xs.t().contiguous().cuda().t())
        off = torch.tensor([0, M // 2, M], dtype=torch.int32).cuda()
        for y in (linear_fp8(xd, (wq, ws), out_dtype=torch.float32),
                  grouped_linear(xd, off, (torch.stack([wq, wq]), torch.stack([ws, ws])), out_dtype=torch.float32)):
            y = y.cpu()
            assert bool(y[2].isnan().all()) and bool(y[4].isnan().all()) and not bool(y[3].isfinite().any())
            assert bool(y[[i for i in range(M) if i not in (2, 3, 4)]].isfinite().all())
