"""GPU test of pw_moe_forward_noalloc (the forward whose scratch is the
library's static device array): through the C ABI, two calls in a row on
one context, the second with a smaller batch, each against pw_moe_forward on
the same inputs (to the layer tolerance; the two may split the down product
differently) and against the float64 oracle; then a batch on the
matrix-core path, and a batch too large for the array, which must fail
cleanly and leave the next call working."""
import pytest
import torch

import synth
from layer_cases import compare_y, cpu_threads, log, make_layer, oracle_y

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    cpu_threads()


def test_noalloc_forward_matches_the_workspace_forward():
    from mixed_precision_weight_page_amd import PagedWeightError
    wl = synth.WORKLOADS["decode_fine"].scaled(name="noalloc", E=32, d=256, F=384, T=64)
    masters = synth.expert_weights(wl)
    layer, _ = make_layer(wl, masters, max_tokens=2048)
    bits = [(3, 4, 8)[e % 3] for e in range(wl.E)]
    layer.quantize_experts(bits)
    for step, T in enumerate((64, 9, 1, 600)):
        x, logits = synth.tokens(wl, T=T, step=step)
        xc, lc = x.cuda(), logits.cuda()
        log(f"noalloc: T={T}")
        y_ws = layer.moe_forward(xc, lc)
        y_st = torch.full((T, wl.d), float("nan"), device="cuda")
        layer.moe_forward_noalloc(xc, lc, y_st)
        torch.cuda.synchronize()
        ref = oracle_y(x, logits, wl, masters, bits)
        compare_y(y_st, y_ws.cpu().double(), f"noalloc vs workspace forward T={T}")
        compare_y(y_st, ref, f"noalloc vs oracle T={T}")


def test_noalloc_refuses_a_batch_larger_than_its_scratch():
    from mixed_precision_weight_page_amd import PagedWeightError
    # 4096 tokens x top-2 at d_model 4096: the partial outputs alone take
    # 128 MiB, more than the static array holds
    wl = synth.WORKLOADS["tiny"].scaled(name="noalloc_big", E=8, d=4096, F=256, k=2, T=4096,
                                        bits=(8, 4, 3, 4, 8, 4, 3, 4))
    masters = synth.expert_weights(wl)
    layer, _ = make_layer(wl, masters, max_tokens=4096)
    layer.quantize_experts(wl.bits)
    x, logits = synth.tokens(wl, T=4096, step=1)
    y = torch.empty((4096, wl.d), device="cuda")
    with pytest.raises(PagedWeightError) as err:
        layer.moe_forward_noalloc(x.cuda(), logits.cuda(), y)
    assert "scratch" in str(err.value)
    x, logits = synth.tokens(wl, T=3, step=2)
    y = torch.empty((3, wl.d), device="cuda")
    layer.moe_forward_noalloc(x.cuda(), logits.cuda(), y)
    torch.cuda.synchronize()
    compare_y(y, oracle_y(x, logits, wl, masters, wl.bits), "noalloc after a refused batch")


def test_noalloc_takes_the_largest_batch_its_scratch_holds():
    """The scratch a forward needs is the workspace without the two counter
    sets of given routes (each cnt [E], act [E] and two more, in 256 bytes):
    the last batch within the array runs, the next one is refused."""
    from mixed_precision_weight_page_amd import PagedMoELayer, PagedWeightError
    E, d, F, k, array = 1024, 128, 128, 1, 64 << 20
    sets = 2 * ((4 * (2 * E + 2) + 255) // 256 * 256)
    need = lambda T: PagedMoELayer(E, d, F, k, max_tokens=T).workspace_bytes() - sets  # noqa: E731
    lo, hi = 1, 1 << 16
    while lo < hi:   # the first batch that does not fit
        mid = (lo + hi) // 2
        lo, hi = (lo, mid) if need(mid) > array else (mid + 1, hi)
    T = lo - 1
    assert need(T) <= array < need(T) + sets
    wl = synth.WORKLOADS["decode_fine"].scaled(name="noalloc_limit", E=E, d=d, F=F, k=k, T=T + 1)
    layer, _ = make_layer(wl, synth.expert_weights(wl), max_tokens=T + 1)
    layer.quantize_experts([(3, 4, 8)[e % 3] for e in range(E)])
    x, logits = (t.cuda() for t in synth.tokens(wl, T=T + 1))
    log(f"noalloc: largest batch, {T} tokens")
    want = layer.moe_forward(x[:T], logits[:T])
    y = torch.full((T, d), float("nan"), device="cuda")
    layer.moe_forward_noalloc(x[:T], logits[:T], y)
    torch.cuda.synchronize()
    compare_y(y, want.cpu().double(), "largest batch")
    with pytest.raises(PagedWeightError, match="scratch"):
        layer.moe_forward_noalloc(x, logits, torch.empty((T + 1, d), device="cuda"))
