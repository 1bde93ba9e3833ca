"""The operators on sampled tokens on masked rows: all but a few entries -inf (or
NaN, or the type's lowest value), and those few far below 0, as behind an
allowed-token mask or where log-probs are given as logits.

Tolerances are those of token_ops_ref.Row for rows of L entries: adding a term
that is 0 is exact, so at most L additions are rounded, and a reference rises at
most L times.  A reference is an entry of the row: with entries within `spread`
of each other an exponent is off by 3 eps (y + spread)."""
import numpy as np
import pytest

import token_ops_ref as R
from test_gpu_token_ops import _check_gradient, _dev, _f64, _logits, _near, _policy, _policy_inputs, _preference

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16"]
LAYOUTS = [24, 140, 320, 620, 800]  # a cluster to a row, then 512, 512, 256 and 192 or 128 threads
LEVELS = (-1.0, -5.0, -8.0, -10.0, -15.0, -20.0, -25.0, -27.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


def _row(x, token, T, entry_bytes):
    row = R.Row(x, token, T, entry_bytes)
    live = row.q > 0
    L, spread = int(live.sum()), float(row.ay[live].max())
    rises = min(np.ceil((row.V * entry_bytes / 32 + 2) / 512), L)
    row.term = 3 * R.EPS * (row.ay + spread) + R.EXP * (rises + 4)
    adds, lnS = L * R.EPS, np.log(row.S)
    row.tol_S = (row.q * row.term).sum() + adds
    row.tol_lnS = row.tol_S + 2 * R.EPS * lnS + R.EPS
    a = abs((x[token] - row.M) / T) if np.isfinite(x[token]) else 0.0
    row.tol_lp = 2 * R.EPS * a + row.tol_lnS + R.EPS * abs(row.lp if np.isfinite(row.lp) else 0.0)
    row.tol_H = row.tol_lnS + (row.q * row.ay * (row.term + adds + row.tol_S + 4 * R.EPS)).sum() + R.EPS * abs(row.H)
    return row


def _masked(rng, n, V, dtype, T, fill):
    """(device logits, values, ids, rows): 24 masked rows (a level and 1, 3 or 100 entries each), the rest not counted."""
    import torch
    lowest = float(torch.finfo(torch.float32 if dtype == "f32" else torch.bfloat16).min)
    x = np.full((n, V), {"inf": -np.inf, "nan": np.nan, "lowest": lowest}[fill], np.float32)
    ids = np.full(n, -1)
    for i in range(24):
        level, count = LEVELS[i % 8], (1, 3, 100)[i // 8]
        at = rng.choice(V - (V // 3 * 2 if i % 2 else 0), count, replace=False) + (V // 3 * 2 if i % 2 else 0)
        x[i, at] = level * T - rng.uniform(0, 3, count) * T
        x[i, at[0]] = level * T
        ids[i] = at[rng.integers(0, count)]
    dev, xs = _logits(x, dtype, 3, 5)
    rows = [_row(xs[i], ids[i], T, 4 if dtype == "f32" else 2) if i < 24 else None for i in range(n)]
    return dev, xs, ids, rows


@pytest.mark.parametrize("fill,T", [("inf", 1.0), ("nan", 1.0), ("lowest", 1.0), ("inf", 0.1), ("nan", 0.1)])
@pytest.mark.parametrize("n", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_score_masked_rows(dtype, n, fill, T):
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(n)
    T = float(np.float32(T))
    dev, _, ids, rows = _masked(rng, n, 70001, dtype, T, fill)
    idd = _dev(ids, np.int32)
    g, gh, zero = rng.standard_normal(n).astype(np.float32), rng.standard_normal(n).astype(np.float32), np.zeros(n)
    for entropy in (False, True):
        lp, h, stats = ls.token_log_probs(dev, idd, temperature=T, entropy=entropy)
        for i in range(24):
            _near(float(lp[i]), rows[i].lp, rows[i].tol_lp, f"lp {i}")
            if entropy:
                _near(float(h[i]), rows[i].H, rows[i].tol_H, f"H {i}")
        for a, b in ((g, zero), (g, gh), (zero, gh)) if entropy else ((g, zero),):
            got = ls.token_log_probs_backward(dev, idd, stats, _dev(a), _dev(b), temperature=T)
            _check_gradient(_f64(got[:24]), rows[:24], a, b, dtype, "gradient")


@pytest.mark.parametrize("n", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_policy_masked_rows(dtype, n):
    rng = np.random.default_rng(n + 1)
    dev, _, ids, rows = _masked(rng, n, 70001, dtype, 1.0, "inf")
    given = _policy_inputs(rng, rows)
    for kw in ({}, {"eta": 0.02}):
        _policy(dev, ids, rows, given, dtype, 1.0, str(kw), **kw)


@pytest.mark.parametrize("dtype", DTYPES)
def test_preference_masked_rows(dtype):
    rng = np.random.default_rng(3)
    for n in (24, 140):
        dev, x, ids, _ = _masked(rng, n, 70001, dtype, 1.0, "inf")
        for ref in (True, False):
            _preference(dev, x, ids, [0, 5, 11, 17, 24], dtype, 1.0, rng, f"{n} rows", ref=ref)


@pytest.mark.parametrize("dtype", DTYPES)
def test_mask_sample_and_score_below_zero(dtype):
    """Log-probs of sampled ids under masks that allow 2 to 60 ids, all below 0: the sampler's own, ratio 1."""
    import logits_sampling_gb300 as ls
    import torch
    n, V = 64, 128256
    rng = np.random.default_rng(4)
    x = (rng.standard_normal((n, V)) - np.linspace(8.0, 30.0, n)[:, None]).astype(np.float32)
    logits, values = _logits(x, dtype)
    words = np.zeros((n, (V + 31) // 32), np.uint32)
    allowed = np.zeros((n, V), bool)
    for i in range(n):
        at = rng.choice(V, 2 + i % 59, replace=False)
        np.bitwise_or.at(words[i], at // 32, np.uint32(1) << (at % 32).astype(np.uint32))
        allowed[i, at] = True
    masked = ls.process_logits(logits, n, allowed_mask=_dev(words.view(np.int32), np.int32))
    prm = ls.SamplingParams.from_host([1.0] * n, [0] * n, [1.0] * n, range(n))
    ids, _, picked = ls.sample_log_probs(masked, n, prm, 0, True, True, want_log_probs=False)
    host = ids.cpu().numpy()
    rows = [_row(np.where(allowed[i], values[i], -np.inf), host[i], 1.0, 4 if dtype == "f32" else 2) for i in range(n)]
    lp, _, _ = ls.token_log_probs(masked, ids)
    one = torch.ones(n, device="cuda")
    _, metrics, _ = ls.policy_loss(masked, ids, one, old_log_probs=picked)
    _, _, fused = ls.policy_loss_grad(masked, ids, one, old_log_probs=picked)
    for i, row in enumerate(rows):
        assert allowed[i, host[i]]
        _near(float(lp[i]), row.lp, row.tol_lp, f"lp {i}")
        for m in (metrics, fused):  # the sampler's own bound on its log-prob is 1e-5
            _near(float(m[i, 3]), 1.0, 1.1e-5 + row.tol_lp, f"ratio {i}")


@pytest.mark.parametrize("T,g_H,level", [(1.0, 1.0, -20.0), (1.0, 1e6, -5.0), (1e-5, 0.02, 0.0), (1e-5, 1.0, 0.0),
                                         (0.01, 65536.0, 0.0), (1e-7, 1.0, 0.0), (1e-37, 1.0, 0.0)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_entropy_gradients_of_masked_entries(dtype, T, g_H, level):
    """Steep entropy gradients: an entry without mass has gradient 0, whatever the slope."""
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(6)
    T, V = float(np.float32(T)), 20001
    for n in (24, 320):
        for fill in (-np.inf, np.nan, -3e38, -50.0 if T < 1e-4 else -np.inf):
            x = np.full((n, V), fill, np.float32)
            ids = np.full(n, -1)
            for i in range(6):
                at = rng.choice(V, 7, replace=False)
                x[i, at] = level - rng.uniform(0, 3, 7) * T
                x[i, at[:2]] = level
                ids[i] = at[i]
            dev, xs = _logits(x, dtype, 3, 5)
            rows = [_row(xs[i], ids[i], T, 4 if dtype == "f32" else 2) for i in range(6)]
            up = np.full(n, g_H)
            idd, gh = _dev(ids, np.int32), _dev(up)
            _, _, stats = ls.token_log_probs(dev, idd, temperature=T, entropy=True)
            grad = _f64(ls.token_log_probs_backward(dev, idd, stats, None, gh, temperature=T)[:6])
            _, fused, _ = ls.policy_loss_grad(dev, idd, _dev(np.zeros(n)), weights=gh, entropy_coef=1.0, temperature=T)
            fused = _f64(fused[:6])
            for got, sign in ((grad, 1.0), (fused, -1.0)):
                _check_gradient(got, rows, np.zeros(n), sign * up, dtype, f"{n} rows of {fill}")


@pytest.mark.parametrize("n,V", [(8, 9001), (8, 70001), (140, 70001), (320, 33001), (620, 70001), (1300, 20011)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_nan_among_masked_entries(dtype, n, V):
    """Rows of -inf but for one allowed id and one NaN, at their ends, next to each other and in shares of their own: the
    NaN has gradient 0, the allowed id log-prob 0 and entropy 0."""
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(V)
    x = np.full((n, V), -np.inf, np.float32)
    ids = np.full(n, -1)
    places = [(0, V - 1), (V - 1, 0), (V // 2, V // 2 + 1), (700, V - 700), (V - 700, 700), (V - 3, V - 2), (1, 0),
              tuple(rng.choice(V, 2, replace=False))]
    for i, (one, nan) in enumerate(places):
        x[i, one], x[i, nan], ids[i] = -12.0, np.nan, one
    dev, _ = _logits(x, dtype, 3, 5)
    idd, g = _dev(ids, np.int32), _dev(rng.standard_normal(n))
    for entropy in (False, True):
        lp, h, stats = ls.token_log_probs(dev, idd, entropy=entropy)
        assert float(lp[:8].abs().max()) <= 2 * R.EXP and (not entropy or float(h[:8].abs().max()) <= 2 * R.EXP)
        back = ls.token_log_probs_backward(dev, idd, stats, g, g if entropy else None)
        _, fused, _ = ls.policy_loss_grad(dev, idd, g, entropy_coef=0.1 * entropy)
        for grad in (back, fused):  # 1 - q of the only entry
            assert torch.isfinite(grad).all() and float(grad.abs().max()) <= float(g.abs().max()) * 8 * R.EXP
            assert not grad.scatter(1, idd.clamp(0).long()[:, None], 0.0).any()
