"""Rows and calls of the operators on sampled tokens at which one part of a row
decides about another: sums far above a warp's reference, NaNs in the units that a
forward pass takes one by one, tokens that have changed since, lists of answers
that overlap."""
import numpy as np
import pytest

import token_ops_ref as R
from test_gpu_token_ops import _dev, _f64, _logits, _near, _normal, _policy, _policy_inputs, _rows, _score

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


@pytest.mark.parametrize("n", [24, 140, 320, 620, 800])
@pytest.mark.parametrize("dtype", DTYPES)
def test_sums_far_above_a_reference(dtype, n):
    """The row's largest entry lies 2^126 above what its warp has seen first, another warp starts just below it."""
    rng = np.random.default_rng(n)
    V = 70001
    x = np.full((n, V), -1.0, np.float32)
    x[:20] += 0.3 * rng.standard_normal((20, V)).astype(np.float32)
    ids = np.full(n, -1)
    for i in range(20):
        x[i, 5] = 87.5
        ids[i] = 30000 + 300 * i
        x[i, ids[i]] = 88.0
    dev, xs = _logits(x, dtype, 2, 6)
    _score(dev, xs, ids, 1.0, dtype, rng, f"{n} rows", some=range(20))
    rows = _rows(xs, ids, 1.0, dtype)
    _policy(dev, ids, rows, _policy_inputs(rng, rows), dtype, 1.0, f"{n} rows")


@pytest.mark.parametrize("n,V", [(6, 9001), (320, 9001), (6, 14000), (700, 14000), (320, 33001), (700, 33001), (6, 70001),
                                 (140, 70001), (1300, 40009)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_single_nans(dtype, n, V):
    """One NaN in a row, wherever it lies: -inf, with gradient 0."""
    rng = np.random.default_rng(V)
    at = [0, 1, 17, V // 2, V - 20, V - 1, V - 700, 700, 5000, V - 5000]
    at += rng.integers(0, V, 14).tolist()
    x = np.zeros((n, V), np.float32)
    x[:24] = _normal(rng, min(n, 24), V)
    ids = np.full(n, -1)
    some = range(min(n, 24))
    for i in some:
        x[i, at[i]] = np.nan
        ids[i] = (at[i] + 3) % V
    for offset in (0, 5):
        dev, xs = _logits(x, dtype, offset, 4)
        _score(dev, xs, ids, 1.0, dtype, rng, f"{n} x {V}", some=some)
        rows = _rows(xs, ids, 1.0, dtype)
        _policy(dev, ids, rows, _policy_inputs(rng, rows), dtype, 1.0, f"{n} x {V}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("op", ["score", "policy", "preference"])
def test_backward_with_tokens_that_have_changed(dtype, op):
    """Ids that have left the vocabulary since the forward call: their rows do not count, and nothing next to a row is
    written."""
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(8)
    for V, n in ((1003, 9), (20001, 7)):
        dev, _ = _logits(_normal(rng, n, V), dtype, 3, 6)
        ids = _dev(rng.integers(0, V, n), np.int32)
        one = _dev(np.ones(n))
        if op == "score":
            stats, back = ls.token_log_probs(dev, ids)[2], lambda i, o: ls.token_log_probs_backward(dev, i, stats, one, out=o)
        elif op == "policy":
            stats, back = ls.policy_loss(dev, ids, one)[2], lambda i, o: ls.policy_loss_backward(dev, i, stats, out=o)
        else:
            stats = ls.preference_loss(dev, ids, _dev([0, 3, n], np.int32))[2]
            back = lambda i, o: ls.preference_loss_backward(dev, i, stats, out=o)  # noqa: E731
        out, _ = _logits(np.zeros((n, V), np.float32), dtype, 3, 6)
        whole = out.as_strided((n * (V + 6) + 4,), (1,), 0)
        assert back(ids, out).any(1).all()
        for far in (-1, -2, -3, V, V + 1, V + 5, V + 12, -2 ** 31, 2 ** 31 - 1):
            whole.fill_(77.0)
            token = np.full(n, far)
            token[1] = int(ids[1])
            got = back(_dev(token, np.int32), out)
            assert (out.as_strided((n, 6), (V + 6, 1), out.storage_offset() + V)[:-1] == 77).all(), far
            assert (whole[:3] == 77).all() and (whole[n * (V + 6) - 3:] == 77).all(), far
            assert got[1].any() and not got[0].any() and not got[2:].any(), far


def test_answers_that_overlap():
    """A list that descends may give a row to two pairs: its pair is bad, and such a row's gradient is the first one's."""
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(9)
    n, V = 900, 64
    dev, _ = _logits(_normal(rng, n, V), "f32")
    ids = _dev(rng.integers(0, V, n), np.int32)
    first = ls.preference_loss(dev, ids, _dev([0, 300, 800, 800, 900], np.int32))
    for bad in ([0, 300, 800, 900, 5, 500, 900], [0, 300, 800, 850, 0, 10, 790, 790, 900]):
        pairs = len(bad) // 2
        for _ in range(20):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            loss, _, stats = ls.preference_loss(dev, ids, _dev(bad, np.int32), error_word=err)
            assert int(err) == ls.LS_ROW_ERR_BAD_OFFSETS and torch.isnan(loss[1]) and torch.isfinite(loss[2:]).all()
            assert torch.equal(loss[0], first[0][0])
            up = torch.arange(1.0, pairs + 1, device="cuda")
            got = ls.preference_loss_backward(dev, ids, stats, up)
            want = ls.preference_loss_backward(dev, ids, first[2], torch.ones(2, device="cuda"))
            assert torch.equal(got[:800], want[:800])


def test_a_loss_without_reference_sums_unrounded_log_probs():
    """1000 rows that allow 1069 ids against 1000 that allow 1070, all alike: their sums differ by 1000 ln(1070 / 1069).

    A row's S is a whole number, and exact; the compensation of the exponentials' mean error is 5.05e-8 (1 - 1 / S) on
    both sides; log2 of 1.044 is off by 2^-28 at most.  So a row's part of the difference is off by less than 1e-8, and
    5e-8 is allowed.  Log-probs rounded to fp32, next to -7, would be off by -2.9e-7 in the one answer's rows and by
    1.3e-7 in the other's.  The loss is u^2 but for 1 / (2 beta)."""
    import logits_sampling_gb300 as ls
    import torch
    n, V = 2000, 2048
    x = torch.full((n, V), -float("inf"), device="cuda")
    x[:1000, :1069] = 0.0
    x[1000:, :1070] = 0.0
    ids = torch.zeros(n, dtype=torch.int32, device="cuda")
    beta = float(np.float32(2.0 ** 20))
    loss, _, _ = ls.preference_loss(x, ids, _dev([0, 1000, 2000], np.int32), beta=beta, loss="ipo")
    u = 1000 * np.log(1070 / 1069)
    got = float(loss[0]) ** 0.5 + 0.5 / beta
    assert abs(got - u) <= 1000 * 5e-8 + 4 * R.EPS * u, (got, u)
