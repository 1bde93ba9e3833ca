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
