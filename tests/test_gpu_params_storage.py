"""GPU checks of a LogitsParams whose tensors change: values in place are what the
next call reads; a tensor that has been resized or given another storage is
refused, for the call would read the memory it had before."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


def _fields():
    import torch
    i32 = {"dtype": torch.int32, "device": "cuda"}
    return {"tokens": torch.tensor([[3, 4, 0, 0], [5, 5, 5, 0]], **i32), "prompt_lens": torch.tensor([0, 0], **i32),
            "seq_lens": torch.tensor([2, 3], **i32), "repetition_penalty": torch.ones(2, device="cuda"),
            "presence_penalty": torch.zeros(2, device="cuda"), "frequency_penalty": torch.ones(2, device="cuda"),
            "bias_offsets": torch.tensor([0, 1, 2], **i32), "bias_ids": torch.tensor([7, 8], **i32),
            "bias_values": torch.tensor([1.0, -1.0], device="cuda")}


def test_values_in_place_are_read_by_the_next_call():
    import torch
    import logits_sampling_gb300 as ls
    f = _fields()
    p = ls.LogitsParams(**f)
    x = torch.zeros(2, 10, device="cuda")
    ls.process_logits(x, 2, p)
    f["tokens"][0, 2] = 9
    f["seq_lens"] += 1
    f["bias_values"] *= 2
    want = torch.zeros(2, 10)
    want[0, [3, 4, 9]] = -1
    want[1, 5], want[1, 0] = -3, -1
    want[0, 7], want[1, 8] = 2, -2
    assert torch.equal(ls.process_logits(x, 2, p).cpu(), want)


@pytest.mark.parametrize("name", list(("tokens", "prompt_lens", "seq_lens", "repetition_penalty", "presence_penalty",
                                       "frequency_penalty", "bias_offsets", "bias_ids", "bias_values")))
@pytest.mark.parametrize("how", ["resize_", "set_", "data", "fewer"])
def test_another_storage_is_refused(name, how):
    import torch
    import logits_sampling_gb300 as ls
    f = _fields()
    p = ls.LogitsParams(**f)
    t = f[name]
    if how == "resize_":
        t.resize_(2, 1 << 20) if name == "tokens" else t.resize_(1 << 20)
    elif how == "set_":
        t.set_(t.clone())
    elif how == "data":
        t.data = t.clone()
    else:
        t.resize_(1, 1) if name == "tokens" else t.resize_(1)
    x = torch.zeros(2, 10, device="cuda")
    with pytest.raises(ValueError, match=f"params' {name} has been resized or given another storage"):
        ls.process_logits(x, 2, p)
