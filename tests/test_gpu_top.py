"""GPU checks of ls_top_log_probs against its definition in 64 bits: ids exact
(ties to the lower id), log-probs and log-sum-exp within the tolerance of their
fp32 arithmetic."""
import numpy as np
import pytest

import row_ops_ref as R

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


def _run(dev, k, T=1.0, gather=None, n=None):
    import torch
    import logits_sampling_gb300 as ls
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = None if gather is None else torch.from_numpy(np.asarray(gather, np.int32)).cuda()
    ids, lp, lse = ls.top_log_probs(dev, k, n=n, temperature=T, gather_indices=g, error_word=err)
    return ids.cpu().numpy(), lp.cpu().numpy(), lse.cpu().numpy(), int(err.item())


def _check(got, x, k, T, where=""):
    ids, lp, lse, _ = got
    for i, row in enumerate(x):
        ref = R.top_row(row, k, T)
        if ref is None:
            assert (ids[i] == -1).all() and np.isnan(lp[i]).all() and np.isnan(lse[i]), (where, i)
            continue
        assert np.array_equal(ids[i], ref[0]), (where, i, ids[i][:8], ref[0][:8])
        fin = np.isfinite(ref[1])
        assert np.array_equal(lp[i][~fin].astype(np.float64), ref[1][~fin]), (where, i)
        off = np.abs(lp[i][fin] - ref[1][fin])
        assert np.all(off <= R.top_tolerance(ref[1][fin])), (where, i, float(off.max()))
        if np.isfinite(ref[2]):
            assert abs(lse[i] - ref[2]) <= R.top_tolerance(ref[2]), (where, i, lse[i], ref[2])
        else:
            assert lse[i] == ref[2], (where, i)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,k", [(1, 1), (2, 2), (5, 3), (31, 31), (300, 256), (1000, 5), (1000, 64), (4097, 20),
                                 (32003, 20), (50000, 256), (128256, 1), (128256, 64), (151936, 20), (262144, 128),
                                 (262144, 256)])
def test_random_rows(dtype, V, k):
    rng = np.random.default_rng(V + k)
    x = R.to_dtype(rng.standard_normal((4, V)) * 3, dtype)
    for T in (1.0, 0.5, 3.0):
        _check(_run(R.device_matrix(x, dtype), k, T), x, k, T, f"T={T}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 7, 40, 200, 700])
def test_batch_sizes(dtype, rows):
    rng = np.random.default_rng(rows)
    x = R.to_dtype(rng.standard_normal((rows, 9001)) * 2, dtype)
    _check(_run(R.device_matrix(x, dtype), 20), x, 20, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("col_off,pad", [(1, 0), (3, 5), (7, 1), (8, 0), (0, 3)])
def test_strides_and_alignments(dtype, col_off, pad):
    rng = np.random.default_rng(col_off)
    x = R.to_dtype(np.round(rng.standard_normal((9, 3001)) * 2), dtype)  # many ties
    _check(_run(R.device_matrix(x, dtype, col_off, pad), 50), x, 50, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,k", [(777, 100), (40000, 200), (200000, 256)])
def test_ties(dtype, V, k):
    """Constant rows, rows of two and of a few values, ties straddling the k-th place."""
    rng = np.random.default_rng(V)
    x = np.zeros((6, V), np.float32)
    x[1] = rng.integers(0, 2, V)
    x[2] = rng.integers(0, 5, V) * -1.5
    x[3, :] = -4.0
    x[3, rng.permutation(V)[:k // 2]] = 1.0
    x[4] = np.arange(V) // (V // 3 + 1)
    x[5] = -0.0
    x[5, ::2] = 0.0
    _check(_run(R.device_matrix(x, dtype), k), R.to_dtype(x, dtype), k, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [777, 60000])
def test_special_values(dtype, V):
    import torch
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((9, V)) * 2).astype(np.float32)
    x[0, ::5] = np.nan
    x[1, [40, 100, 700]] = np.inf
    x[2, :] = -np.inf
    x[3, :] = np.nan
    x[4, :] = -np.inf
    x[4, [5, 776, 600]] = [1.0, -3.0, 1.0]
    x[5, :] = float(torch.finfo(torch.bfloat16).min)
    x[5, 7] = -1e30
    x[6, ::2] = -np.inf
    x[7, :] = np.inf
    x[8, :700] = np.nan
    x[8, 700:720] = -np.inf
    x = R.to_dtype(x, dtype)
    got = _run(R.device_matrix(x, dtype), 30)
    _check(got, x, 30, 1.0)
    assert got[3] == ls.LS_ROW_ERR_NO_FINITE


@pytest.mark.parametrize("dtype", DTYPES)
def test_long_tails(dtype):
    """Values spread over orders of magnitude: most exponentials underflow."""
    rng = np.random.default_rng(6)
    x = R.to_dtype(-np.exp(rng.random((4, 20000)) * 20), dtype)
    for T in (0.01, 1.0, 1000.0):
        got = _run(R.device_matrix(x, dtype), 40, T)
        _check(got, x, 40, T, f"T={T}")


def test_gather_and_bad_rows():
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(9)
    x = R.to_dtype(rng.standard_normal((20, 5000)) * 3, "bf16")
    gather = np.array([3, 19, 0, 25, -1, 7, 7, 12])
    ids, lp, lse, err = _run(R.device_matrix(x, "bf16"), 9, gather=gather)
    assert err == ls.LS_ROW_ERR_BAD_GATHER
    assert (ids[3:5] == -1).all() and np.isnan(lp[3:5]).all() and np.isnan(lse[3:5]).all()
    good = [0, 1, 2, 5, 6, 7]
    _check((ids[good], lp[good], lse[good], 0), x[gather[good]], 9, 1.0)


def test_offsets_past_32_bits():
    import torch
    V, rows = 262144, 16640
    x = torch.zeros((rows, V), dtype=torch.bfloat16, device="cuda")
    x[-2:] = torch.randn(2, V, device="cuda").to(torch.bfloat16)
    host = x[-2:].float().cpu().numpy()
    _check(_run(x, 20, gather=[rows - 2, rows - 1]), host, 20, 1.0)
    ids, lp, lse, _ = _run(x, 3)
    _check((ids[-2:], lp[-2:], lse[-2:], 0), host, 3, 1.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_largest_vocab(dtype):
    import logits_sampling_gb300 as ls
    V = ls.row_ops_max_vocab(ls.LS_DTYPE_BF16)
    assert V == ls.row_ops_max_vocab(ls.LS_DTYPE_F32) >= 1 << 22
    rng = np.random.default_rng(0)
    x = R.to_dtype(rng.standard_normal((2, V)) * 3, dtype)
    _check(_run(R.device_matrix(x, dtype, 1, 1), 100), x, 100, 1.0)
    with pytest.raises(ls.LSError):
        ls.top_log_probs(R.device_matrix(np.zeros((1, V + 1)), dtype), 3)


def test_same_bits_every_time_on_any_stream():
    import torch
    import logits_sampling_gb300 as ls
    x = (torch.randn(300, 32000, device="cuda") * 3).to(torch.bfloat16)
    a = ls.top_log_probs(x, 20)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = ls.top_log_probs(x, 20, stream=s)
    s.synchronize()
    for u, v in zip(a, b):
        assert torch.equal(u, v)
    out = [torch.zeros_like(t) for t in a]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ls.top_log_probs(x, 20, out_ids=out[0], out_log_probs=out[1], out_lse=out[2])
    g.replay()
    torch.cuda.synchronize()
    for u, v in zip(a, out):
        assert torch.equal(u, v)


def test_agrees_with_the_sampler():
    """The first id is the greedy id; the log-probs are those that ls_log_probs writes."""
    import torch
    import logits_sampling_gb300 as ls
    x = (torch.randn(40, 32000, device="cuda") * 3).to(torch.bfloat16)
    ids, lp, _ = ls.top_log_probs(x, 10)
    assert torch.equal(ids[:, 0], ls.argmax(x))
    n = 40
    rows = ls.log_probs(x, ls.SamplingParams.from_host([1.0] * n, [0] * n, [1.0] * n, [0] * n))
    assert float((rows.gather(1, ids.long()) - lp).abs().max()) <= 1e-4
