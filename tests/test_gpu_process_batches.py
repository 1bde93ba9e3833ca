"""GPU checks of ls_process_logits where a history reaches its kernels in more
than one batch of ids: rows of mostly distinct ids, each row of its own, against
the definition in 64 bits, between the two choices of kernels and between
repetitions, bit for bit."""
import numpy as np
import pytest

import row_ops_ref as R

pytestmark = pytest.mark.gpu
V = 33000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()
    yield
    ls.set_process_policy(0)


def _forced(policy, *args):
    import torch
    import logits_sampling_gb300 as ls
    ls.set_process_policy(policy)
    out = ls.process_logits(*args)
    ls.set_process_policy(0)
    return out.view(torch.int32 if out.dtype == torch.float32 else torch.int16)


def _case(rng, rows, length, biases):
    """x, params and a function that gives row i's definition."""
    import torch
    import logits_sampling_gb300 as ls
    x = R.to_dtype(rng.standard_normal((rows, V)) * 3, "f32")
    tokens = np.stack([rng.permutation(V)[:length] for _ in range(rows)]).astype(np.int32)
    tokens[:, 5::50] = tokens[:, :1]  # one id over and over
    prompt = rng.integers(0, length, rows).astype(np.int32)
    rho, pres, freq = (R.to_dtype(v, "f32") for v in (1 + rng.random(rows), rng.random(rows), rng.random(rows) * 0.5))
    bias = [dict(zip(rng.permutation(V)[:biases].tolist(), R.to_dtype(rng.standard_normal(biases), "f32").tolist()))
            for _ in range(rows)] if biases else None

    def dev(v, t):
        return torch.from_numpy(np.ascontiguousarray(v, t)).cuda()

    off = {} if bias is None else {
        "bias_offsets": dev(np.arange(rows + 1) * biases, np.int32), "bias_ids": dev([list(b) for b in bias], np.int32).view(-1),
        "bias_values": dev([list(b.values()) for b in bias], np.float32).view(-1)}
    params = ls.LogitsParams(tokens=dev(tokens, np.int32), prompt_lens=dev(prompt, np.int32),
                             seq_lens=dev(np.full(rows, length), np.int32), repetition_penalty=dev(rho, np.float32),
                             presence_penalty=dev(pres, np.float32), frequency_penalty=dev(freq, np.float32), **off)
    return x, params, lambda i: R.process_row(x[i], tokens[i], prompt[i], float(rho[i]), float(pres[i]), float(freq[i]),
                                              bias[i] if bias else None)


# one batch of 4096 ids; an id more; two full batches; the most that one table takes, with and without biases; past it
@pytest.mark.parametrize("length,biases", [(4096, 0), (4097, 0), (8192, 0), (8832, 0), (8192, 640), (8193, 640)])
def test_full_batches_of_distinct_ids(length, biases):
    import torch
    rng = np.random.default_rng(length + biases)
    rows = 300
    x, params, definition = _case(rng, rows, length, biases)
    dev = torch.from_numpy(x).cuda()
    got = _forced(2, dev, rows, params)
    for _ in range(10):
        assert torch.equal(_forced(2, dev, rows, params), got)
    assert torch.equal(_forced(1, dev, rows, params), got)
    out = got.view(torch.float32).cpu().numpy()
    for i in range(rows):
        y, touched, tol = definition(i)
        assert np.array_equal(out[i][~touched], x[i][~touched]), (i, "untouched entries")
        assert R.within(out[i][touched], y[touched], tol[touched], "f32").all(), i
