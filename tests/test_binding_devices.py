"""The sampler's calls run on the device that holds their data, whichever is
current: tensors that claim a device and have no storage stand for those of a
second GPU."""
import contextlib

import pytest
import torch

import logits_sampling_gb300 as ls


class Claimed(torch.Tensor):
    """A tensor with a shape, a type and a device, and no memory."""

    @staticmethod
    def __new__(cls, shape, dtype=torch.float32, device=1):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=f"cuda:{device}")

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"a call computes with {func}")


class Stopped(Exception):
    pass


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from logits_sampling_gb300 import build as b
    b.build()


X = Claimed((4, 1000))
CANDIDATES = Claimed((2, 2), torch.int32)
CALLS = {
    "sample": (X, lambda s: ls.sample(X, 4, None, 0, True, True, stream=s)),
    "sample_speculative": (X, lambda s: ls.sample_speculative(X, 1, 2, 1, None, 0, True, True, stream=s)),
    "log_probs": (X, lambda s: ls.log_probs(X, None, stream=s)),
    "sample_log_probs": (X, lambda s: ls.sample_log_probs(X, 4, None, 0, True, True, stream=s)),
    "sample_log_probs_noalloc": (X, lambda s: ls.sample_log_probs_noalloc(X, 4, None, 0, True, True, stream=s)),
    "sample_device_step": (X, lambda s: ls.sample_device_step(X, 4, None, Claimed((1,), torch.int64), True, True,
                                                              stream=s)),
    "argmax": (X, lambda s: ls.argmax(X, stream=s)),
    "verify_chain": (CANDIDATES, lambda s: ls.verify_chain(CANDIDATES, Claimed((4,), torch.int32), stream=s)),
    "sample_verify": (X, lambda s: ls.sample_verify(X, CANDIDATES, None, 0, True, True, stream=s)),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_a_call_takes_the_current_stream_of_its_data_and_its_device(monkeypatch, name):
    data, call = CALLS[name]
    asked = []

    def current_stream(device=None):
        asked.append(device)
        return "that device's stream"

    def make_current(stream):
        assert stream == "that device's stream"
        raise Stopped

    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.setattr(torch.cuda, "stream", make_current)
    with pytest.raises(Stopped):
        call(None)
    assert asked == [data.device]


@pytest.mark.parametrize("name", list(CALLS))
def test_a_stream_of_another_device_is_refused(monkeypatch, name):
    class Stream:
        device, cuda_stream = torch.device("cuda:0"), 0

    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    with pytest.raises(ValueError, match="stream is on cuda:0, cuda:1 holds the data"):
        CALLS[name][1](Stream())
