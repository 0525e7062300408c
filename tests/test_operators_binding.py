"""Host-only checks of the Python binding of the calls around the expert
layer. No call here touches a GPU."""
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
