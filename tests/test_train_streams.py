"""Calls of the training operators on a given stream: what they refuse there."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

from allreduce_compatible_gradient_amd import train  # noqa: E402


class Stream:
    """A stream's outside, for a machine without a GPU."""

    def __init__(self, index):
        self.cuda_stream, self.device = 1, torch.device("cuda", index)


def test_a_refusal_on_a_stream_keeps_its_error(monkeypatch):
    """Host tensors among the arguments, which the operator refuses, are not
    recorded on the stream: that would raise an error of its own."""
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    given = torch.zeros(3), train.Act8.empty(3, 8, "cpu"), None
    with pytest.raises(ValueError, match="weight must be"):
        with train._Elsewhere(torch.device("cuda", 0), Stream(0), given):
            raise ValueError("weight must be a tensor on cuda:0")


@pytest.mark.gpu
def test_refusals_on_another_stream():
    x = torch.randn(4, 64, device="cuda")
    w, host8 = torch.ones(64), train.Act8.empty(4, 64, "cpu")
    side = torch.cuda.Stream()
    for stream in (None, side, side.cuda_stream):
        for call in (lambda: train.gqt_layer_norm(x, w, stream=stream),
                     lambda: train.gqt_layer_norm(x, save_x=host8, stream=stream),
                     lambda: train.gqt_act8_save(x, out=host8, stream=stream),
                     lambda: train.gqt_gelu_backward(x, host8, stream=stream),
                     lambda: train.gqt_weight_grad(x, host8, stream=stream)):
            with pytest.raises(ValueError):
                call()


def test_a_stream_of_another_device_is_refused():
    """It would switch the device, and the work would then run on that of the
    tensors, on a stream that the caller did not name."""
    with pytest.raises(ValueError, match="stream"):
        train._Elsewhere(torch.device("cuda", 0), Stream(1), ())
    assert train._Elsewhere(torch.device("cuda", 1), Stream(1), ()).stream.cuda_stream == 1
