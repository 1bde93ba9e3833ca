"""The calls on logits rows refuse tensors and streams of another device than the
logits' before any CUDA call: tensors that claim a device and have no storage
stand for those of a second GPU."""
import pytest
import torch

import logits_sampling_gb300 as ls


class Claimed(torch.Tensor):
    """A tensor with a shape, a type and a device, and no memory."""

    @staticmethod
    def __new__(cls, shape, dtype=torch.float32, device=0):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device=f"cuda:{device}")

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise AssertionError(f"a call computes with {func}")


class Stream:
    stream_id, device_index, device_type = 0, 1, 1


N, V, K = 4, 1000, 8
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from logits_sampling_gb300 import build as b
    b.build()


def _arguments():
    """Per call: what it needs, and every further tensor that it may be given, all on device 0."""
    x, ids, lp = Claimed((N, V)), Claimed((N, K), I32), Claimed((N, K))
    vec, ivec, word = Claimed((N,)), Claimed((N,), I32), Claimed((1,), I32)
    return {
        "process_logits": ({"logits": x, "n": N},
                           {"gather_indices": ivec, "token_to_request_index": ivec, "row_lens": ivec,
                            "allowed_mask": Claimed((N, 32), I32), "mask_index": ivec, "out": x, "error_word": word}),
        "top_log_probs": ({"logits": x, "k": K},
                          {"gather_indices": ivec, "out_ids": ids, "out_log_probs": lp, "out_lse": vec,
                           "error_word": word}),
        "distill_loss": ({"logits": x, "teacher_ids": ids, "teacher_log_probs": lp},
                         {"weights": vec, "out": vec, "out_stats": Claimed((N, 8)), "error_word": word}),
        "distill_loss_backward": ({"logits": x, "teacher_ids": ids, "teacher_log_probs": lp, "stats": Claimed((N, 8))},
                                  {"grad_loss": vec, "weights": vec, "out": x}),
        "distill_loss_grad": ({"logits": x, "teacher_ids": ids, "teacher_log_probs": lp},
                              {"weights": vec, "out_loss": vec, "out_grad": x, "error_word": word}),
    }


def _elsewhere(t):
    return Claimed(tuple(t.shape), t.dtype, 1)


@pytest.mark.parametrize("call", list(_arguments()))
def test_tensors_of_another_device_are_refused(call):
    need, more = _arguments()[call]
    for name in (n for n in (*need, *more) if n != "logits" and isinstance({**need, **more}[n], torch.Tensor)):
        given = {**need, **more}
        given[name] = _elsewhere(given[name])
        with pytest.raises(ValueError, match=f"{name} is on cuda:1, the logits are on cuda:0"):
            getattr(ls, call)(**given)


@pytest.mark.parametrize("call", list(_arguments()))
def test_streams_of_another_device_are_refused(call):
    need, _ = _arguments()[call]
    with pytest.raises(ValueError, match="stream is on cuda:1, the logits are on cuda:0"):
        getattr(ls, call)(**need, stream=Stream())


def test_parameters_of_another_device_are_refused():
    def fields(device):
        return {"tokens": Claimed((N, 16), I32, device), "seq_lens": Claimed((N,), I32, device),
                "repetition_penalty": Claimed((N,), torch.float32, device)}

    with pytest.raises(ValueError, match="params is on cuda:1, the logits are on cuda:0"):
        ls.process_logits(Claimed((N, V)), N, ls.LogitsParams(**fields(1)))
    for name in fields(0):
        with pytest.raises(ValueError, match="different devices"):
            ls.LogitsParams(**{**fields(0), name: fields(1)[name]})
