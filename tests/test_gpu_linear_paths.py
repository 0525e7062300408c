"""GPU tests of pw_linear on each of its kernels for up to 64 tokens (rows
straight into registers, and through the waves' LDS rings: fewer and more
pieces of K than a ring holds, one to four waves, whole and ragged ends), with
the bounds of test_gpu_linear.py, and of long sums on every kernel.

Long sums are exact: the operands are whole numbers of 1 to 32 with either
sign, which bf16 and fp16 hold, so every sum of products stays a whole number
below 14336 * 32^2 < 2^24 in any order, and an fp32 sum rounds nowhere. A
product left out, taken twice, or a partial sum in fewer bits shows."""
import pytest
import torch

from layer_cases import cpu_threads, log
from test_gpu_linear import DT, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cpu_threads()


# by blocks of 16 tokens and 32 weight rows: 1 and 2 blocks of tokens with
# rows on either side of 8192, 3 and 4 with rows that fill the GPU once and
# not; the last N is no multiple of a block
FEW = [(1, 8203), (16, 8203), (17, 4200), (32, 8190), (32, 8200), (33, 2800), (48, 4201), (64, 4200), (64, 9000)]


@pytest.mark.parametrize("K", [8, 64, 200, 264, 520, 1096])
@pytest.mark.parametrize("M,N", FEW)
def test_few_tokens_through_rings(M, N, K):
    run(M, N, K, "none", "bf16", "f32", bias=True)
    run(M, (N + 1) // 2, K, "swiglu", "f16", "f16", bias=True, residual=True, pads=(8, 16, 4, 4))


# the same token blocks with rows of odd length; the ring of loads wraps from
# 16 pieces of 64 on
@pytest.mark.parametrize("K", [65, 700, 1437])
@pytest.mark.parametrize("M,N", [(5, 8200), (17, 4100), (32, 4133), (33, 2800), (48, 2801), (64, 2100)])
def test_few_tokens_with_odd_rows(M, N, K):
    run(M, N, K, "silu", "f16", "f32", bias=True, pads=(1, 0, 0, 0))
    run(M, (N + 1) // 2, K, "swiglu", "bf16", "bf16", residual=True, pads=(0, 3, 1, 0))


# sizes for every kernel, its name beside them
LONG = [(1, 256, 14336), (16, 512, 8192), (5, 300, 8191),        # rows into registers, the last of odd length
        (16, 8200, 4096), (32, 4200, 2056), (64, 9000, 1096),    # rings of each wave
        (48, 2800, 2049),                                        # registers, odd rows, several token blocks
        (200, 300, 8192), (1100, 2300, 2048), (2100, 2900, 1096),  # tiles of 64 x 64, 128 x 128, 256 x 128
        (4000, 2800, 1096), (4000, 3900, 1096),                  # 192 x 256 and 256 x 256
        (300, 200, 8191)]                                        # tiles of odd rows


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", LONG)
def test_long_sums_are_exact(M, N, K, dtype):
    from mixed_precision_weight_page_amd import linear
    gen = torch.Generator().manual_seed(M + N + K)
    whole = lambda *s: (torch.randint(1, 33, s, generator=gen) * (2 * torch.randint(0, 2, s, generator=gen) - 1)).to(DT[dtype])  # noqa: E731
    x, w = whole(M, K), whole(N, K)
    log(f"long sums {M}x{N}x{K} {dtype}")
    y = linear(x.cuda(), w.cuda(), out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), x.double() @ w.double().t())
