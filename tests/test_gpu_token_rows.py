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
