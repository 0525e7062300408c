"""Host-only checks of the Python binding of the calls around the expert
layer. No call here touches a GPU."""
import ctypes
import os
import threading

import pytest
import torch

from mixed_precision_weight_page_amd import pagedweight as pwb


class Stream:
    """Stands in for a torch stream of a device."""
    def __init__(self, handle, device=0):
        self.cuda_stream, self.device = handle, torch.device("cuda", device)


def test_which_stream_a_call_runs_on(monkeypatch):
    default, side = Stream(0), Stream(0x1000)
    here = [default]
    made = []

    def external(handle):
        made.append(handle)
        return Stream(handle)

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: here[0])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: default)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    # on the default stream: its handle, None and the stream itself are the current one
    for s in (None, 0, default):
        assert pwb._other_stream(s) is None
    assert pwb._other_stream(side) is side
    assert pwb._other_stream(0x1000).cuda_stream == 0x1000 and made == [0x1000]
    # on another one: 0 is the default stream, never a new one
    here[0] = side
    assert pwb._other_stream(0) is default and made == [0x1000]
    assert pwb._other_stream(default) is default
    for s in (None, 0x1000, side):
        assert pwb._other_stream(s) is None
    # the default streams of two devices share the handle 0
    here[0] = default
    other = Stream(0, device=1)
    assert pwb._other_stream(other) is other


needs_lib = pytest.mark.skipif(not os.path.exists(pwb.library_path()), reason="library not built")
FAKE, ODD = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 1)


def c_linear(x=FAKE, w=FAKE, r=None, y=FAKE, desc=True, **kw):
    """pw_linear on pointers that a refused call never reads."""
    d = pwb.LinearDesc(**{**dict(M=4, N=8, K=16, in_dtype=2, out_dtype=2, act=0, ldx=16, ldw=16, ldr=8, ldy=8), **kw})
    return pwb.lib().pw_linear(ctypes.byref(d) if desc else None, x, w, None, r, y, None)


@needs_lib
def test_every_refusal_of_linear_says_why():
    L = pwb.lib()
    for bad, word in ((dict(desc=False), b"description"), (dict(M=-1), b"M = -1"), (dict(K=(1 << 29) + 1), b"2^29"),
                      (dict(in_dtype=0), b"type 0"), (dict(out_dtype=3), b"got 3"), (dict(act=7), b"activation 7"),
                      (dict(ldx=15), b"rows of x are 15"), (dict(ldw=15), b"rows of w are 15"), (dict(ldy=7), b"rows of y are 7"),
                      (dict(r=FAKE, ldr=7), b"rows of residual are 7"), (dict(ldx=1 << 22), b"2^22"), (dict(x=None), b"null x"),
                      (dict(w=None), b"null w"), (dict(y=None), b"null y"), (dict(x=ODD), b"aligned")):
        assert c_linear(**bad) == -1, bad
        assert word in L.pw_last_error(None), (bad, L.pw_last_error(None))
    # the message is the calling thread's own
    other = []
    t = threading.Thread(target=lambda: other.extend([c_linear(act=9), L.pw_last_error(None)]))
    t.start()
    t.join()
    assert other[0] == -1 and b"activation 9" in other[1]
    assert b"aligned" in L.pw_last_error(None)


@needs_lib
def test_the_binding_passes_the_reason_on(monkeypatch):
    # everything up to the library's own checks, as if the tensors were on a GPU
    monkeypatch.setattr(pwb, "_here", lambda t, name: (0, None))
    monkeypatch.setattr(pwb, "_on_gpu", lambda t, dev, name: None)
    x, w = torch.zeros(1, 16, dtype=torch.bfloat16).expand(4, 16), torch.zeros(8, 16, dtype=torch.bfloat16)
    with pytest.raises(pwb.PagedWeightError, match="rows of x are 0 elements apart"):
        pwb.linear(x, w)


@needs_lib
def test_tensors_that_require_a_gradient_are_refused(monkeypatch):
    monkeypatch.setattr(pwb, "_here", lambda t, name: (0, None))
    layer = pwb.PagedMoELayer(8, 128, 128, 2, max_tokens=4)
    x, w = torch.zeros(2, 16).bfloat16().requires_grad_(), torch.zeros(8, 16).bfloat16()
    logits = torch.zeros(2, 8, requires_grad=True)
    tokens = torch.zeros(2, 128).bfloat16().requires_grad_()
    calls = (lambda: pwb.linear(x, w), lambda: layer.route_gated(logits),
             lambda: layer.moe_forward_routed(tokens, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)))
    for call in calls:
        with pytest.raises(ValueError, match="forward only"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):   # on to the next check
            call()


@needs_lib
def test_a_residual_that_is_y_has_its_rows():
    assert c_linear(r=FAKE, y=FAKE, ldr=8, ldy=9) == -1
    assert b"residual is y" in pwb.lib().pw_last_error(None)
    assert c_linear(r=FAKE, y=FAKE, ldr=9, ldy=8) == -1
    # a single row has no distance to a next one (refused for its alignment only)
    assert c_linear(r=ODD, y=ODD, M=1, ldr=8, ldy=9) == -1
    assert b"aligned" in pwb.lib().pw_last_error(None)


@needs_lib
def test_products_that_one_launch_cannot_cover_are_refused():
    for kw in (dict(M=1 << 24, N=1 << 24, ldr=1 << 24, ldy=1 << 24),                  # aligned tiles
               dict(M=1 << 20, N=1 << 20, K=15, ldx=15, ldw=15, ldy=1 << 20),        # rows of any alignment
               dict(M=1, N=1 << 30, K=15, ldx=15, ldw=15), dict(M=(1 << 31) - 1),    # one token; most tokens
               dict(M=1, N=1 << 30, K=512, ldx=512, ldw=512), dict(M=1 << 30, N=1, K=1, ldx=1, ldw=1, ldy=1)):
        assert c_linear(**kw) == -1, kw
        assert b"2^32" in pwb.lib().pw_last_error(None), kw
