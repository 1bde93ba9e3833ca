"""The operators on logits rows on a host without a GPU: every call refuses bad
arguments before any CUDA call, and the 64-bit definitions that the GPU tests
compare with hold against differences and closed forms."""
import ctypes

import numpy as np
import pytest

import row_ops_ref as R

P = ctypes.c_void_p
FAKE, FAR = P(0x10000), P(0x10000000)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from logits_sampling_gb300 import build as b
    b.build()
    from logits_sampling_gb300 import _row_ops
    return _row_ops._lib()


def test_process_refusals(lib):
    from logits_sampling_gb300._row_ops import _LogitsParams

    def call(logits=FAKE, dt=1, rows=4, V=40, stride=40, n=4, gather=None, t2r=None, params=None, lens=None, mask=None,
             mask_rows=4, mask_stride=2, index=None, out=FAR, out_stride=40):
        return lib.ls_process_logits(logits, dt, rows, V, stride, n, gather, t2r,
                                     None if params is None else ctypes.byref(params), lens, mask, mask_rows,
                                     mask_stride, index, out, out_stride, None, None)

    def params(**kw):
        s = _LogitsParams(num_requests=4)
        for k, v in kw.items():
            setattr(s, k, v)
        return s

    fake = 0x10000
    assert call(n=0) == 0
    for kw in ({"n": -1}, {"logits": None}, {"dt": 5}, {"V": 0}, {"stride": 39}, {"out": None}, {"out_stride": 39},
               {"n": 5}, {"logits": P(0x10001)}, {"out": P(0x10000001)}, {"rows": 0, "gather": FAKE},
               {"logits": P(0x10002), "dt": 0}, {"V": 0x7FFFFFFF, "stride": 0x7FFFFFFF, "out_stride": 0x7FFFFFFF},
               {"mask": FAKE, "mask_rows": 3}, {"mask": FAKE, "mask_stride": 1},
               {"mask": FAKE, "mask_rows": 0, "index": FAKE},
               {"out": FAKE, "out_stride": 48}, {"out": FAKE, "gather": FAKE}, {"out": P(0x10010)},
               {"params": params(num_requests=0)}, {"params": params(num_requests=3)},
               {"params": params(tokens=fake, token_capacity=8, token_stride=7, seq_lens=fake)},
               {"params": params(tokens=fake, token_capacity=-1, token_stride=7, seq_lens=fake)},
               {"params": params(tokens=fake, token_capacity=8, token_stride=8)},
               {"params": params(bias_offsets=fake, bias_count=-1)},
               {"params": params(bias_offsets=fake, bias_count=3, bias_ids=fake)}):
        assert call(**kw) == 1, kw
    big = 1 << 30  # lengths whose strides through them would pass 32 bits
    assert call(params=params(tokens=fake, token_capacity=big, token_stride=big, seq_lens=fake)) == 2
    assert call(params=params(bias_offsets=fake, bias_count=big, bias_ids=fake, bias_values=fake)) == 2


def test_process_policy_values(lib):
    for bad in (-1, 3, 8):
        assert lib.ls_set_process_policy(bad) == 1, bad
    for good in (1, 2, 0):
        assert lib.ls_set_process_policy(good) == 0, good


def test_top_refusals(lib):
    def call(logits=FAKE, dt=1, rows=4, V=400, stride=400, n=4, gather=None, k=4, T=1.0, ids=FAR, lp=FAR):
        return lib.ls_top_log_probs(logits, dt, rows, V, stride, n, gather, k, T, ids, lp, None, None, None)

    assert call(n=0) == 0
    for kw in ({"n": -1}, {"logits": None}, {"dt": 5}, {"V": 0}, {"stride": 399}, {"n": 5}, {"k": 0}, {"k": 257},
               {"k": 41, "V": 40}, {"T": 0.0}, {"T": -1.0}, {"T": float("inf")}, {"T": float("nan")}, {"ids": None},
               {"lp": None}, {"logits": P(0x10001)}):
        assert call(**kw) == 1, kw
    assert call(V=1 << 24, stride=1 << 24) == 2


def test_distill_refusals(lib):
    from logits_sampling_gb300._row_ops import _Teacher

    def teacher(ids=0x10000, lp=0x10000, stride=8, k=8):
        return ctypes.byref(_Teacher(ids, lp, stride, k))

    def loss(logits=FAKE, dt=1, V=400, stride=400, n=4, t=teacher(), T=1.0, tail=2, out=FAR, stats=None):
        return lib.ls_distill_loss(logits, dt, V, stride, n, t, T, tail, None, out, stats, None, None)

    def back(logits=FAKE, dt=1, V=400, stride=400, n=4, t=teacher(), T=1.0, tail=2, stats=FAKE, out=FAR, out_stride=400):
        return lib.ls_distill_loss_backward(logits, dt, V, stride, n, t, T, tail, None, stats, None, out, out_stride,
                                            None)

    def both(logits=FAKE, dt=1, V=400, stride=400, n=4, t=teacher(), T=1.0, tail=2, loss_=FAKE, out=FAR,
             out_stride=400):
        return lib.ls_distill_loss_grad(logits, dt, V, stride, n, t, T, tail, None, loss_, out, out_stride, None, None)

    common = [{"n": -1}, {"logits": None}, {"dt": 5}, {"V": 0}, {"stride": 399}, {"T": 0.0}, {"T": float("nan")},
              {"T": float("inf")}, {"tail": 3}, {"tail": -1}, {"t": None}, {"t": teacher(ids=None)},
              {"t": teacher(lp=None)}, {"t": teacher(k=0)}, {"t": teacher(k=257, stride=257)}, {"t": teacher(stride=7)},
              {"out": None}]
    for f in (loss, back, both):
        assert f(n=0) == 0
        assert f(V=1 << 24, stride=1 << 24, **({} if f is loss else {"out_stride": 1 << 24})) == 2
        for kw in common:
            assert f(**kw) == 1, (f.__name__, kw)
    assert loss(stats=P(0x10004)) == 1
    assert back(stats=None) == 1 and back(stats=P(0x10004)) == 1
    assert both(loss_=None) == 1
    for f in (back, both):
        for kw in ({"out_stride": 399}, {"out": FAKE, "out_stride": 408}, {"out": P(0x10010)}, {"out": P(0x10000001)}):
            assert f(**kw) == 1, (f.__name__, kw)


def test_binding_refusals():
    import torch
    import logits_sampling_gb300 as ls
    x = torch.zeros(2, 10)
    with pytest.raises(ValueError):
        ls.process_logits(x)  # not on a GPU
    with pytest.raises(ValueError):
        ls.LogitsParams()
    with pytest.raises(ValueError):
        ls.LogitsParams(tokens=torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        ls.top_log_probs(x, 3)
    with pytest.raises(TypeError):
        ls.top_log_probs(x.to(torch.float16), 3)
    with pytest.raises(ValueError):
        ls.distill_loss(x, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3))


def test_max_vocab_without_a_device_or_with_one(lib):
    import torch
    for dt in (0, 1):
        v = lib.ls_row_ops_max_vocab(dt)
        assert v >= 262144 if torch.cuda.is_available() else v == 0


@pytest.mark.parametrize("tail", ["drop", "renorm", "bucket"])
def test_distill_definition_against_differences(tail):
    rng = np.random.default_rng(0)
    V, k, T = 40, 6, 1.7
    x = rng.standard_normal(V) * 2
    ids = rng.permutation(V)[:k]
    lp = np.log(rng.dirichlet(np.ones(k + 3))[:k])
    _, _, grad, _ = R.distill_row(x, ids, lp, T, tail, 0.7, 1.3)
    for j in range(V):
        d = np.zeros(V)
        d[j] = 1e-5
        up, dn = (R.distill_row(x + s * d, ids, lp, T, tail, 0.7)[0] for s in (1, -1))
        assert abs((up - dn) / 2e-5 * 1.3 - grad[j]) < 1e-8  # h^2 of third differences and 1e-16 / h


def test_distill_definition_closed_forms():
    x = np.log(np.array([0.5, 0.25, 0.125, 0.125]))
    lp = np.log(np.array([0.5, 0.25]))
    for tail, want in (("drop", 0.0), ("bucket", 0.0), ("renorm", np.log(1 / 0.75))):
        loss, _, grad, _ = R.distill_row(x, [0, 1], lp, 1.0, tail)
        assert abs(loss - want) < 1e-15, tail
    assert np.abs(R.distill_row(x, [0, 1], lp, 1.0, "bucket")[2]).max() < 1e-15


def test_process_definition_closed_form():
    y, touched, _ = R.process_row([2.0, -2.0, 1.0, 0.5], [0, 1, 1, 0, 1], 2, 2.0, 0.5, 0.25, {2: 1.0},
                                  np.array([1, 1, 1, 0], bool))
    assert y.tolist() == [2.0 / 2 - 0.25 - 0.5, -4.0 - 0.5 - 0.5, 2.0, -np.inf]
    assert touched.tolist() == [True] * 4
