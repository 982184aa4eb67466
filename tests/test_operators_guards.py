"""The binding's device and stream guards (CPU: torch's are replaced): a call that is
refused while they are being set up leaves the current device and stream as they
were."""
import pytest
import torch

from matrix_optimizers_amd import operators as O


class Guards:
    """Stands in for torch.cuda.device and torch.cuda.stream: what is entered and not left."""

    def __init__(self, monkeypatch):
        self.open = []
        monkeypatch.setattr(O.torch.cuda, "current_device", lambda: 0)
        monkeypatch.setattr(O.torch.cuda, "device", lambda d: self.guard("device", d))
        monkeypatch.setattr(O.torch.cuda, "stream", lambda s: self.guard("stream", s))

    def guard(self, *what):
        outer = self

        class G:
            def __enter__(self):
                if isinstance(what[1], Broken):
                    raise RuntimeError("no such stream")
                outer.open.append(what)

            def __exit__(self, *exc):
                assert outer.open.pop() == what
        return G()


class Broken:
    """A stream whose guard cannot be entered."""
    cuda_stream = 5


@pytest.mark.parametrize("stream,error", [("x", ValueError), (object(), TypeError), (Broken(), RuntimeError)])
def test_a_refused_stream_leaves_no_guard(monkeypatch, stream, error):
    g = Guards(monkeypatch)
    monkeypatch.setattr(O.torch.cuda, "ExternalStream", lambda h, device: stream)
    with pytest.raises(error):
        with O._On(torch.device("cuda", 1), stream):
            pass
    assert g.open == []


def test_guards_are_left_in_order(monkeypatch):
    g = Guards(monkeypatch)

    class S:
        cuda_stream = 7
    monkeypatch.setattr(O.torch.cuda, "ExternalStream", lambda h, device: S())
    with pytest.raises(KeyError):
        with O._On(torch.device("cuda", 1), 7) as on:
            assert [w[0] for w in g.open] == ["device", "stream"] and on.handle == 7
            raise KeyError
    assert g.open == []
