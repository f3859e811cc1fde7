"""The device and stream switches around a call, with fake guards (no GPU):
whatever goes wrong on the way in, the caller's device and stream are as before."""
import pytest
import torch

import integer_only_quantized_b200 as ia

DEV = torch.device("cuda", 1)


class Fakes:
    """Current device and stream, and how they change."""

    def __init__(self, monkeypatch, bad_stream_guard=False):
        self.device, self.stream, self.made = 0, "own", []
        outer = self

        class Guard:
            field = None

            def __init__(self, value):
                self.value = value.index if isinstance(value, torch.device) else value

            def __enter__(self):
                if self.field == "stream" and bad_stream_guard:
                    raise RuntimeError("no such stream")
                self.old = getattr(outer, self.field)
                setattr(outer, self.field, self.value)

            def __exit__(self, *exc):
                setattr(outer, self.field, self.old)

        class Stream:
            def __init__(self, handle, device=None):
                self.cuda_stream, self.device = handle, device
                outer.made.append(handle)

        class Current:
            cuda_stream = property(lambda self: getattr(outer.stream, "cuda_stream", outer.stream))

        monkeypatch.setattr(torch.cuda, "device", type("D", (Guard,), {"field": "device"}))
        monkeypatch.setattr(torch.cuda, "stream", type("S", (Guard,), {"field": "stream"}))
        monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
        monkeypatch.setattr(torch.cuda, "Stream", Stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Current())

    def untouched(self):
        return self.device == 0 and self.stream == "own"


@pytest.mark.parametrize("stream", ["seven", object(), [3]])
def test_a_stream_of_the_wrong_type_leaves_the_device(monkeypatch, stream):
    f = Fakes(monkeypatch)
    with pytest.raises((TypeError, ValueError)):
        with ia._On(DEV, stream):
            pass
    assert f.untouched()


def test_a_stream_that_cannot_be_entered_leaves_the_device(monkeypatch):
    f = Fakes(monkeypatch, bad_stream_guard=True)
    with pytest.raises(RuntimeError):
        with ia._On(DEV, 77):
            pass
    assert f.untouched()


def test_a_stream_of_another_device(monkeypatch):
    f = Fakes(monkeypatch)
    with pytest.raises(ValueError):
        with ia._On(DEV, torch.cuda.Stream(5, torch.device("cuda", 0))):
            pass
    assert f.untouched()


def test_device_and_stream_of_a_call(monkeypatch):
    f = Fakes(monkeypatch)

    class Handle:  # of another library
        cuda_stream = 78

    for stream, handle in ((None, "own"), (77, 77), (Handle(), 78), (torch.cuda.Stream(79, DEV), 79)):
        with ia._On(DEV, stream) as h:
            assert h == handle and f.device == 1
        assert f.untouched()
        with pytest.raises(KeyError):
            with ia._On(DEV, stream):
                raise KeyError
        assert f.untouched()
