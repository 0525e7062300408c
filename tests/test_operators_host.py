"""Host-only checks of the calls around the expert layer (pw_route_gated,
pw_moe_forward_routed, pw_linear): the C ABI's refusals, with pointers that
are never dereferenced, and the Python binding's. No call here touches a
GPU."""
import ctypes
import os

import pytest
import torch

from mixed_precision_weight_page_amd import pagedweight as pwb

PW_OK, INVALID, WORKSPACE, STATE = 0, -1, -6, -7
FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(pwb.library_path()):
        pytest.skip("library not built")
    return pwb.lib()


@pytest.fixture()
def ctx(L):
    desc = pwb.LayerDesc(num_experts=12, d_model=128, d_ff=256, top_k=4, renorm=0, max_tokens=8, master_dtype=0)
    c = ctypes.c_void_p()
    assert L.pw_create(ctypes.byref(desc), ctypes.byref(c)) == PW_OK
    yield c
    L.pw_destroy(c)


def gate(L, ctx, T=4, dtype=0, ld=12, logits=FAKE, bias=None, mask=None, ids=FAKE, g=FAKE, counts=None, desc=True, **kw):
    d = pwb.GateDesc(**{**dict(score=0, n_group=1, topk_group=1, group_top2=0, renorm=0, scale=1.0), **kw})
    return L.pw_route_gated(ctx, ctypes.byref(d) if desc else None, logits, dtype, ld, bias, mask, T, ids, g, counts, None)


def test_gate_refusals(L, ctx):
    assert gate(L, None) == INVALID
    assert gate(L, ctx, desc=False) == INVALID
    for bad in (dict(T=-1), dict(T=9), dict(score=2), dict(n_group=0), dict(n_group=5), dict(n_group=4, topk_group=0),
                dict(n_group=4, topk_group=5), dict(n_group=4, topk_group=1), dict(n_group=12, topk_group=3),
                dict(group_top2=2), dict(renorm=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(dtype=3),
                dict(dtype=-1), dict(ld=11), dict(logits=None), dict(ids=None), dict(g=None), dict(logits=ODD),
                dict(bias=ODD), dict(ids=ODD), dict(g=ODD), dict(counts=ODD)):
        assert gate(L, ctx, **bad) == INVALID, bad
        assert L.pw_last_error(ctx)
    # nothing to do, nothing touched
    assert gate(L, ctx, T=0, logits=None, ids=None, g=None) == PW_OK


def test_more_groups_than_the_gate_takes(L):
    desc = pwb.LayerDesc(num_experts=130, d_model=128, d_ff=128, top_k=1, renorm=0, max_tokens=8, master_dtype=0)
    c = ctypes.c_void_p()
    assert L.pw_create(ctypes.byref(desc), ctypes.byref(c)) == PW_OK
    assert gate(L, c, ld=130, n_group=65, topk_group=2) == INVALID
    L.pw_destroy(c)


def test_routed_refusals(L, ctx):
    call = lambda T=2, x=FAKE, ids=FAKE, g=FAKE, r=None, y=FAKE, dt=0: L.pw_moe_forward_routed(ctx, x, ids, g, T, r, y, dt, None)  # noqa: E731
    assert L.pw_moe_forward_routed(None, FAKE, FAKE, FAKE, 1, None, FAKE, 0, None) == INVALID
    for bad in (dict(T=-1), dict(T=9), dict(dt=1), dict(dt=3), dict(ids=None), dict(g=None), dict(ids=ODD), dict(g=ODD), dict(r=ODD)):
        assert call(**bad) == INVALID, bad
    assert call() == WORKSPACE
    n = L.pw_workspace_bytes(ctx)
    assert L.pw_bind_workspace(ctx, FAKE, n) == PW_OK
    assert call() == STATE          # no pages
    assert call(T=0) == STATE


def linear(L, x=FAKE, w=FAKE, bias=None, r=None, y=FAKE, desc=True, **kw):
    d = pwb.LinearDesc(**{**dict(M=4, N=8, K=16, in_dtype=2, out_dtype=2, act=0, ldx=16, ldw=16, ldr=8, ldy=8), **kw})
    return L.pw_linear(ctypes.byref(d) if desc else None, x, w, bias, r, y, None)


def test_linear_refusals(L):
    for bad in (dict(desc=False), dict(M=-1), dict(N=-1), dict(K=-1), dict(N=(1 << 30) + 1), dict(K=(1 << 29) + 1),
                dict(in_dtype=0), dict(in_dtype=3), dict(out_dtype=3), dict(act=-1), dict(act=7), dict(ldx=15),
                dict(ldw=15), dict(ldy=7), dict(r=FAKE, ldr=7), dict(ldx=1 << 22), dict(ldw=1 << 22), dict(x=None),
                dict(w=None), dict(y=None), dict(x=ODD), dict(w=ODD), dict(bias=ODD), dict(r=ODD), dict(y=ODD),
                dict(out_dtype=0, y=ctypes.c_void_p((1 << 20) + 2)), dict(ldx=-16)):
        assert linear(L, **bad) == INVALID, bad
    assert linear(L, M=0, x=None, y=None) == PW_OK
    assert linear(L, N=0, w=None, y=None) == PW_OK


def test_binding_refusals():
    x, w = torch.zeros(2, 16).bfloat16(), torch.zeros(8, 16).bfloat16()
    with pytest.raises(ValueError, match="act"):
        pwb.linear(x, w, act="tanh")
    with pytest.raises(ValueError, match="2-d"):
        pwb.linear(x[0], w)
    with pytest.raises(ValueError, match="gate as up"):
        pwb.linear(x, w[:7], act="swiglu")
    with pytest.raises(ValueError, match="CUDA"):
        pwb.linear(x, w)
    layer = pwb.PagedMoELayer(8, 128, 128, 2, max_tokens=4)
    for kw in (dict(score="tanh"), dict(group_score="sum")):
        with pytest.raises(ValueError, match="score"):
            layer.route_gated(torch.zeros(2, 8), **kw)
    with pytest.raises(ValueError, match="logits"):
        layer.route_gated(torch.zeros(8))
    with pytest.raises(ValueError, match="CUDA"):
        layer.route_gated(torch.zeros(2, 8))
    with pytest.raises(ValueError, match=r"\[T, k\]"):
        layer.moe_forward_routed(torch.zeros(2, 128).bfloat16(), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3))
    with pytest.raises(ValueError, match="out_dtype"):
        layer.moe_forward_routed(torch.zeros(2, 128).bfloat16(), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2),
                                 out_dtype=torch.float16)
