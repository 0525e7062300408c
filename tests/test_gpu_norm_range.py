"""GPU tests of pw_rms_norm where h w, r or their fp32 order would leave fp32's
range although y does not: y and scales within 2^-18 of float64 (the sum's
and r's error as in test_gpu_norm.py, two products; in fp64 far less), and half
a step of y's type. Codes are those of the exact h w: with weights that are
powers of two, or h and weights of 16 bits, fp32 and fp64 give the same."""
import math

import pytest
import torch

from layer_cases import log
from product_cases import DT, E4M3, nearest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(x, w, eps, residual=None):
    from mixed_precision_weight_page_amd import rms_norm
    h = x.float() if residual is None else (x.float() + residual.float()).to(residual.dtype)
    d = h.double()
    T, n = d.shape
    r = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + torch.tensor(eps).double())   # eps in fp32
    z = d * w.double()
    args = (x.cuda(), w.cuda(), eps, None if residual is None else residual.cuda())
    first = (lambda got: got) if residual is None else (lambda got: got[0])
    for out in (torch.float32, torch.bfloat16):
        y = first(rms_norm(*args, out_dtype=out)).cpu().double()
        want = z * r
        tol = want.abs() * (2.0 ** -18 + torch.finfo(out).eps / 2) + torch.finfo(out).tiny
        assert bool(((y - want).abs() <= tol).all()), (out, float(((y - want).abs() / tol).max()))
    got = first(rms_norm(*args, out_dtype=E4M3))
    q, s = got.q.float().cpu().double(), got.scale.cpu().double()
    for b in range(-(-n // 128)):
        cols = slice(128 * b, 128 * b + 128)
        m = z[:, cols].abs().amax(dim=1, keepdim=True).clamp_min(2.0 ** -100)
        assert torch.equal(q[:, cols], nearest((448.0 * z[:, cols] / m).float()))
        want = (m * r)[:, 0] / 448
        # below 2^-126 fp32 has steps of 2^-149: half of one more (a block of zeros has m r = 2^-100 / 3e38)
        assert bool(((s[:, b] - want).abs() <= 2.0 ** -18 * want + 2.0 ** -150).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 130, 640, 700, 2051, 20000])
def test_rows_near_the_top(n, dtype):
    """|h| up to 3e38 and weights above one."""
    gen = torch.Generator().manual_seed(n)
    x = (torch.rand(5, n, generator=gen) * 6e38 - 3e38).clamp(-3e38, 3e38)
    x[1, : n // 2] *= 1e-30
    x[2] *= 1e-19            # squares fit, their sum does not
    x[3, 1:] = 0
    w = 2.0 ** torch.randint(-3, 12, (n,), generator=gen).float()
    log(f"norm {n} {dtype} near the top")
    check(x.to(DT[dtype]), w, 1e-6)
    check(x.to(DT[dtype]), w.bfloat16(), 0.0)
    half = x.to(DT[dtype]) / 2
    check(half, w, 1e-6, half.clone())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [8, 130, 640, 2051])
def test_rows_of_subnormals(n, dtype):
    """With eps = 0 a root mean square of 1e-40 has a reciprocal beyond fp32."""
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(4, n, generator=gen) * 1e-38
    x[1] *= 1e-2
    x[2] = 0
    x[2, n // 2] = 2.0 ** -133
    x[3] *= 1e8
    log(f"norm {n} {dtype} of subnormals")
    check(x.to(DT[dtype]), torch.ones(n), 0.0)


@pytest.mark.parametrize("n", [8, 136, 700, 5000])
def test_weights_that_carry_h_out_of_range(n):
    """Ordinary sums of squares, but h w over- or underflows before r is applied."""
    gen = torch.Generator().manual_seed(n)
    x = torch.randn(6, n, generator=gen)
    w = 2.0 ** torch.randint(0, 3, (n,), generator=gen).float()
    x = x * torch.tensor([1e12, 1e16, 1.0, 1e-9, 1e17, 1e5])[:, None]
    log(f"norm {n}, weights of 2^90 and 2^-100")
    check(x, w * 2.0 ** 90, 1e-6)
    check(x, w * 2.0 ** -100, 0.0)


def test_infinities_stay_as_they_were():
    """A row with an infinity: NaN there and zeros beside it (r = 1 / sqrt(inf) = 0), in 8 bits with
    scales m r: inf 0 = NaN for its block, 0 for the row's others; other rows are not touched."""
    from mixed_precision_weight_page_amd import rms_norm
    x = torch.full((3, 300), 3e38)
    x[1, 17] = math.inf
    w = torch.full((300,), 2.0)
    y = rms_norm(x.cuda(), w.cuda()).cpu()
    assert bool(y[1, 17].isnan()) and int(y[1].isnan().sum()) == 1 and bool((y[1].nan_to_num(0.0) == 0).all())
    assert bool(((y[[0, 2]] - 2.0).abs() <= 2.0 ** -17).all())
    q = rms_norm(x.cuda(), w.cuda(), out_dtype=E4M3)
    assert bool((q.q.float()[[0, 2]] == 448.0).all()) and bool(q.q.float()[1, 17].isnan())
    assert bool(q.scale[1, 0].isnan()) and bool((q.scale[1, 1:] == 0).all())
    w[5] = math.inf
    q = rms_norm(x[:1].cuda(), w.cuda(), out_dtype=E4M3)
    assert bool(q.q.float()[0, 5].isnan()) and bool((q.q.float()[0, 6:128] == 0).all()) and bool((q.q.float()[0, 128:] == 448.0).all())
    assert bool(q.scale[0, 0].isinf()) and bool(q.scale[0, 1:].isfinite().all())
