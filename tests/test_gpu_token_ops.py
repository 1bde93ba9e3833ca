"""GPU checks of the operators on sampled tokens against their definitions in 64
bits, and of their gradients against differences of the losses."""
import numpy as np
import pytest

import token_ops_ref as R

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


def _dev(v, t=np.float32):
    import torch
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v, t)).cuda()


def _f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def _logits(x, dtype, offset=0, pad=0):
    """(device logits, float64 values as the device holds them): rows start `offset` entries in, `pad` entries apart."""
    import torch
    n, V = x.shape
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    buf = torch.full((n * (V + pad) + offset + 1,), 77.0, dtype=t, device="cuda")
    dev = buf[offset:offset + n * (V + pad)].view(n, V + pad)[:, :V]
    dev.copy_(torch.from_numpy(x.astype(np.float32)))
    return dev, _f64(dev)


def _rows(x, ids, T, dtype, counted=None):
    return [R.Row(x[i], ids[i], T, 4 if dtype == "f32" else 2)
            if 0 <= ids[i] < x.shape[1] and (counted is None or counted[i]) else None for i in range(len(x))]


def _near(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    tol = np.broadcast_to(np.asarray(tol, np.float64), want.shape)
    # past the largest fp32 number, 2^128 (1 - 2^-24), a value in fp32 is infinite
    want = np.where(np.abs(want) > 2.0 ** 128 * (1 - 2.0 ** -24), np.copysign(np.inf, want), want)
    with np.errstate(invalid="ignore"):
        ok = (np.isnan(got) & np.isnan(want)) | (got == want) | (np.abs(got - want) <= tol + R.TINY)
    if not ok.all():
        at = np.unravel_index(np.argmin(ok), ok.shape)
        raise AssertionError(f"{what}: {np.sum(~ok)} off, first at {at}: got {got[at]}, want {want[at]} +- {tol[at]}")


def _check_gradient(got, rows, g_lp, g_H, dtype, what, tol_g=None):
    for i, row in enumerate(rows):
        if row is None or (g_lp[i] == 0 and g_H[i] == 0):
            assert not got[i].any(), f"{what}: row {i} counts nothing"
            continue
        d, tol = row.gradient(g_lp[i], g_H[i])
        if tol_g is not None and row.some:
            one = np.zeros(row.V)
            one[row.token] = 1.0
            tol = tol + tol_g[i] * np.abs(one - row.q) / row.T
        _near(got[i], d, tol + R.HALF_STEP[dtype] * (np.abs(d) + tol), f"{what}, row {i}")


def _score(dev, x, ids, T, dtype, rng, what="", some=None):
    """token_log_probs with and without entropies, and every kind of gradient (of rows `some`: all)."""
    import logits_sampling_gb300 as ls
    n = len(ids)
    some = range(n) if some is None else some
    rows = [None] * n
    for i in some:
        rows[i] = _rows(x[i:i + 1], ids[i:i + 1], T, dtype)[0]
    idd = _dev(ids, np.int32)
    lp0, none, stats0 = ls.token_log_probs(dev, idd, temperature=T)
    lp1, h, stats1 = ls.token_log_probs(dev, idd, temperature=T, entropy=True)
    assert none is None and stats0.shape == (n, ls.TOKEN_STATS)
    for i in some:
        row = rows[i]
        for lp in (lp0, lp1):
            _near(float(lp[i]), 0.0 if row is None else row.lp, 0.0 if row is None or not row.some else row.tol_lp,
                  f"{what} lp {i}")
        _near(float(h[i]), 0.0 if row is None else row.H, 0.0 if row is None or not row.some else row.tol_H, f"{what} H {i}")
    g_lp, g_H = rng.standard_normal(n).astype(np.float32), rng.standard_normal(n).astype(np.float32)
    zero = np.zeros(n)
    for stats, a, b in ((stats0, g_lp, None), (stats1, g_lp, g_H), (stats1, None, g_H)):
        got = ls.token_log_probs_backward(dev, idd, stats, _dev(a), _dev(b), temperature=T)
        at = list(some)
        _check_gradient(_f64(got[at]), [rows[i] for i in at], (zero if a is None else a)[at], (zero if b is None else b)[at],
                        dtype, f"{what} gradient")


def _normal(rng, n, V, scale=3.0):
    return (rng.standard_normal((n, V)) * scale).astype(np.float32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 7, 15, 16, 17, 33, 255, 1000, 1023, 4097, 8191, 16385])
def test_score_sizes(dtype, V):
    rng = np.random.default_rng(V)
    for n, T, offset, pad in ((1, 1.0, 0, 0), (5, 0.7, 1, 3), (3, 1.9, 5, 0)):
        dev, x = _logits(_normal(rng, n, V), dtype, offset, pad)
        ids = rng.integers(0, V, n)
        ids[0] = (0, V - 1, V // 2)[n % 3]
        _score(dev, x, ids, T, dtype, rng, f"{n} x {V}, T {T}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,V", [(1, 128256), (3, 262144), (700, 1001), (200, 32003), (9, 400001), (1300, 9001),
                                 (400, 40003)])
def test_score_batches(dtype, n, V):
    rng = np.random.default_rng(n + V)
    dev, x = _logits(_normal(rng, n, V), dtype, 3, 5)
    _score(dev, x, rng.integers(0, V, n), 1.0, dtype, rng, f"{n} x {V}", some=range(0, n, max(1, n // 100)))


def _special(rng, dtype, V):
    """20 rows of special values, and their tokens."""
    import torch
    lowest = float(torch.finfo(torch.float32 if dtype == "f32" else torch.bfloat16).min)
    x = _normal(rng, 20, V)
    ids = rng.integers(0, V, 20)
    x[0, rng.integers(0, V, 900)] = np.nan
    x[1, rng.integers(0, V, 2900)] = -np.inf
    x[2, rng.integers(0, V, 2900)] = lowest
    x[3] = -np.inf
    x[3, 77] = 2.0
    ids[3] = 77
    x[4] = lowest
    x[5] = -np.inf                      # nothing left
    x[6] = np.nan                       # nothing left
    x[7, [5, 900, 3000]] = np.inf
    ids[7] = 900
    x[8, [5, 900]] = np.inf
    ids[8] = 6
    x[9, ids[9]] = -np.inf
    x[10, ids[10]] = np.nan
    x[11] += 20000.0
    x[12] -= 20000.0
    x[13] = 1.5
    x[14, ids[14]] = 60.0               # all but certain
    x[15] *= 1e4
    x[16] *= 1e30
    x[17] *= 1e-30
    x[18] = lowest
    x[18, 3] = 0.0
    x[19, ::2] = np.nan
    x[19, 1::2] = -np.inf
    x[19, 2] = 1.0
    return x, ids


@pytest.mark.parametrize("dtype", DTYPES)
def test_score_special_rows(dtype):
    """NaN, infinities, the type's lowest value as a mask, rows that leave one entry or none, far and equal values."""
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(5)
    V = 3001
    x, ids = _special(rng, dtype, V)
    dev, xs = _logits(x, dtype, 2, 6)
    for T in (1.0, 0.05, 30.0):
        _score(dev, xs, ids, T, dtype, rng, f"T {T}")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ls.token_log_probs(dev, _dev(ids, np.int32), entropy=True, error_word=err)
    assert int(err) == ls.LS_ROW_ERR_NO_FINITE
    err.zero_()
    keep = [i for i in range(20) if i not in (5, 6)]
    ls.token_log_probs(dev[keep], _dev(ids[keep], np.int32), error_word=err)
    assert int(err) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [20, 140, 320, 620, 800])
def test_score_special_long_rows(dtype, n):
    """The same in rows of many stages, for each layout of a batch; and rows whose maximum is far above what the first
    stages hold, below their reference, or all in one place."""
    rng = np.random.default_rng(50)
    V = 70001
    x = _normal(rng, n, V)
    x[:20], ids20 = _special(rng, dtype, V)
    ids = rng.integers(0, V, n)
    ids[:20] = ids20
    if n > 20:
        x[20, 60000:60010] = 33.0               # sums far above 1
        x[21, 69000] = 90.0                     # past what a sum against the first stage may hold
        x[22, :50000] = -np.inf                 # nothing in the first stages
        x[23, :] = -np.inf
        x[23, 69990:] = -300.0                  # far below the reference of a warp that has none
        x[24, :50000] = -200.0
        x[25, 100] = 500.0
        ids[20:26] = 60003, 69000, 60000, 69995, 60001, 100
    dev, xs = _logits(x, dtype, 2, 6)
    some = list(range(26)) if n > 20 else list(range(20))
    _score(dev, xs, ids, 1.0, dtype, rng, f"{n} rows", some=some)


@pytest.mark.parametrize("T", [1e-30, 1e-7, 1e9, 1e25, 3e38])
@pytest.mark.parametrize("dtype", DTYPES)
def test_score_far_temperatures(dtype, T):
    rng = np.random.default_rng(6)
    dev, x = _logits(_normal(rng, 4, 501), dtype)
    ids = x.argmax(1)
    _score(dev, x, ids, np.float32(T).astype(np.float64), dtype, rng, f"T {T}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_that_do_not_count(dtype):
    """Ids outside the vocabulary and weights of 0: nothing is read (NaN stays unseen), outputs and gradients are 0."""
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(7)
    V, n = 1003, 8
    dev, x = _logits(_normal(rng, n, V), dtype, 1, 4)
    ids = rng.integers(0, V, n)
    ids[1], ids[3], ids[4] = -1, V, -100
    dev[[1, 3, 4, 6]] = float("nan")
    idd = _dev(ids, np.int32)
    nan = torch.full((n,), float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids6 = ids.copy()
    ids6[6] = -1
    _score(dev, x, ids6, 1.0, dtype, rng)
    lp, h, stats = ls.token_log_probs(dev, _dev(ids6, np.int32), entropy=True, error_word=err)
    grad = ls.token_log_probs_backward(dev, _dev(ids6, np.int32), stats, nan, nan)
    skipped = [1, 3, 4, 6]
    for t in (lp, h, grad):
        assert not t[skipped].any()
    w = np.ones(n, np.float32)
    w[6] = 0.0
    adv = nan.clone()
    how = {"weights": _dev(w), "old_log_probs": nan, "ref_log_probs": nan, "kl_coef": 0.1, "entropy_coef": 0.1}
    loss, metrics, stats = ls.policy_loss(dev, idd, adv, error_word=err, **how)
    loss2, grad2, metrics2 = ls.policy_loss_grad(dev, idd, adv, error_word=err, **how)
    grad = ls.policy_loss_backward(dev, idd, stats, nan)
    for t in (loss, metrics, grad, loss2, grad2, metrics2):
        assert not t[skipped].any() and torch.isnan(t[[0, 2, 5, 7]]).any(-1).all()
    off = torch.tensor([1, 3, 5], dtype=torch.int32, device="cuda")  # rows 0 and 5 on are in no answer
    dev[[0, 5, 7]] = float("nan")
    loss, ratios, stats = ls.preference_loss(dev, idd, off, weights=_dev(w), error_word=err)
    assert torch.isfinite(loss).all() and float(ratios[1]) == 0.0
    grad = ls.preference_loss_backward(dev, idd, stats)
    assert grad[2].any() and not grad[[0, 1, 3, 4, 5, 6, 7]].any()
    assert int(err) == 0


# -- the policy loss ------------------------------------------------------------


def _policy_inputs(rng, rows, spread=0.5):
    n = len(rows)
    lp = np.array([0.0 if r is None or not np.isfinite(r.lp) else r.lp for r in rows])
    d = rng.standard_normal(n) * spread
    for border in (0.8, 1.2, 1.28, 3.0):  # a ratio next to a border may fall on either side
        d = np.where(np.abs(d - np.log(border)) < 1e-3, np.log(border) + 2e-3, d)
    return {"A": rng.standard_normal(n).astype(np.float32), "old": (lp - d).astype(np.float32),
            "ref": (lp + rng.standard_normal(n) * 0.4).astype(np.float32),
            "w": rng.uniform(0.5, 1.5, n).astype(np.float32), "up": rng.standard_normal(n).astype(np.float32)}


def _policy(dev, ids, rows, given, dtype, T, what="", old=True, ref=True, w=True, lo=0.2, hi=0.28, dual=0.0, beta=0.05,
            kl="k3", eta=0.0, entropy=False, keep=lambda i: True):
    import logits_sampling_gb300 as ls
    import torch
    n = len(rows)
    idd = _dev(ids, np.int32)
    how = {"old_log_probs": _dev(given["old"]) if old else None, "ref_log_probs": _dev(given["ref"]) if ref else None,
           "weights": _dev(given["w"]) if w else None, "temperature": T, "clip_low": lo, "clip_high": hi,
           "dual_clip": dual, "kl_coef": beta, "kl": kl, "entropy_coef": eta, "entropy": entropy}
    A, up = _dev(given["A"]), _dev(given["up"])
    loss, metrics, stats = ls.policy_loss(dev, idd, A, **how)
    grad = ls.policy_loss_backward(dev, idd, stats, up, temperature=T)
    plain = ls.policy_loss_backward(dev, idd, stats, temperature=T)
    loss2, grad2, metrics2 = ls.policy_loss_grad(dev, idd, A, **how)
    f = [float(np.float32(v)) for v in (lo, hi, dual, beta, eta)]
    want = []
    for i, row in enumerate(rows):
        if row is None or not keep(i):
            want.append(None)
            continue
        want.append(R.policy_row(row, float(given["A"][i]), float(given["old"][i]) if old else None,
                                 float(given["ref"][i]) if ref else None, float(given["w"][i]) if w else 1.0, f[0], f[1],
                                 f[2], f[3], kl, f[4]))
    for i, r in enumerate(want):
        if r is None:
            continue
        row = rows[i]
        for got, m in ((loss, metrics), (loss2, metrics2)):
            _near(float(got[i]), r[0], r[4] + 2 * R.EPS * abs(r[0]) if row.some else 0, f"{what} loss {i}")
            if row.some:
                _near(_f64(m[i]), (r[1][0], r[1][1] if entropy or eta else 0.0, r[1][2], r[1][3]),
                      (row.tol_lp, row.tol_H, r[5], r[6]), f"{what} metrics {i}")
    some = [i for i in range(n) if want[i] is not None]
    picked = [rows[i] for i in some]
    for got, u in ((grad, given["up"]), (plain, np.ones(n)), (grad2, np.ones(n))):
        _check_gradient(_f64(got)[some], picked, [want[i][2] * u[i] for i in some], [want[i][3] * u[i] for i in some], dtype,
                        f"{what} gradient", [abs(u[i]) * want[i][7] for i in some])
    return torch.equal(loss, loss2) and torch.equal(plain, grad2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 3, 16, 250, 1001, 8200, 32003])
def test_policy_sizes(dtype, V):
    rng = np.random.default_rng(V)
    for n, T, kw in ((1, 1.0, {}), (13, 0.7, {"eta": 0.03, "kl": "k2"}), (40, 1.3, {"dual": 3.0, "kl": "k1", "entropy": True})):
        dev, x = _logits(_normal(rng, n, V), dtype, n % 7, n % 5)
        ids = rng.integers(0, V, n)
        rows = _rows(x, ids, T, dtype)
        _policy(dev, ids, rows, _policy_inputs(rng, rows), dtype, T, f"{n} x {V}", **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kw", [{"old": False}, {"ref": False, "beta": 0.0}, {"w": False}, {"old": False, "ref": False, "beta": 0.0},
                                {"beta": 0.0, "eta": 0.1}, {"hi": float("inf")}, {"lo": 0.0, "hi": 0.0}, {"lo": 1.0},
                                {"dual": 1.0}, {"dual": 2.5, "eta": -0.2}, {"beta": -0.3, "kl": "k2"}])
def test_policy_terms(dtype, kw):
    rng = np.random.default_rng(11)
    V, n = 2051, 48
    dev, x = _logits(_normal(rng, n, V), dtype, 4, 2)
    ids = np.argsort(-x, 1)[np.arange(n), rng.integers(0, 30, n)]
    rows = _rows(x, ids, 1.0, dtype)
    given = _policy_inputs(rng, rows, 0.8)
    given["A"][::9] = 0.0
    _policy(dev, ids, rows, given, dtype, 1.0, str(kw), **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,V", [(700, 1000), (161, 32000), (6, 262144), (310, 16391), (130, 400001), (311, 90001)])
@pytest.mark.parametrize("eta", [0.0, 0.01])
def test_policy_batches(dtype, n, V, eta):
    rng = np.random.default_rng(n)
    dev, x = _logits(_normal(rng, n, V), dtype, *((0, 0) if V % 2 == 0 else (1, 2)))
    ids = rng.integers(0, V, n)
    at = set(range(0, n, max(1, n // 50)))
    rows = _rows(x, ids, 1.0, dtype, [i in at for i in range(n)])
    _policy(dev, ids, rows, _policy_inputs(rng, rows), dtype, 1.0, f"{n} x {V}", eta=eta)


@pytest.mark.parametrize("dtype", DTYPES)
def test_policy_special_rows(dtype):
    """Excluded tokens (log-probs of -inf on either side), ratios past every bound, rows without an entry."""
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(12)
    V, n = 1100, 16
    x = _normal(rng, n, V)
    ids = rng.integers(0, V, n)
    for i in (0, 1, 2, 3, 4):
        x[i, ids[i]] = -np.inf
    x[9] = -np.inf
    x[10, ::3] = -np.inf
    x[10, ids[10]] = 1.0
    x[11] = np.inf
    x[12] = np.nan
    dev, xs = _logits(x, dtype, 1, 1)
    rows = _rows(xs, ids, 1.0, dtype)
    given = _policy_inputs(rng, rows)
    given["A"][[0, 5, 7]], given["A"][[1, 6, 8]], given["A"][12] = 1.5, -1.5, 0.0
    given["old"][2] = given["ref"][0] = given["ref"][1] = given["ref"][2] = given["old"][3] = -np.inf
    given["ref"][3] = given["ref"][4] = -np.inf
    given["old"][[5, 6]] = -200.0       # ratios past what fp32 holds
    given["old"][[7, 8]] = 50.0
    for kw in ({}, {"dual": 3.0, "eta": 0.1}, {"kl": "k2"}, {"kl": "k1"}):
        # 6: an infinite loss unless dual_clip bounds it; its gradient is not a number
        _policy(dev, ids, rows, given, dtype, 1.0, str(kw), keep=lambda i: i != 6 or "dual" in kw, **kw)
    given["ref"][13] = -np.inf           # a reference that excludes what was sampled: infinite KL
    idd, how = _dev(ids, np.int32), {"ref_log_probs": _dev(given["ref"]), "kl_coef": 0.1}
    for kl, slope in (("k1", 1.0), ("k2", np.inf), ("k3", 1.0)):
        loss, m, _ = ls.policy_loss(dev, idd, _dev(given["A"]), kl=kl, **how)
        assert float(loss[13]) == np.inf and float(m[13, 2]) == np.inf
    loss, _, _ = ls.policy_loss(dev, idd, _dev(given["A"]))
    assert np.isnan(float(loss[9])) and np.isnan(float(loss[12]))  # no entry left, whatever the advantage


# -- the preference loss --------------------------------------------------------


def _preference(dev, x, ids, offsets, dtype, T, rng, what="", ref=True, w=None, **how):
    import logits_sampling_gb300 as ls
    n, P = len(ids), len(offsets) // 2
    inside = [offsets[0] <= i < offsets[-1] for i in range(n)]
    rows = _rows(x, ids, T, dtype, [k and (w is None or w[i] != 0) for i, k in enumerate(inside)])
    lp = [None if r is None else r.lp for r in rows]
    refs = np.array([0.0 if v is None or not np.isfinite(v) else v for v in lp]) + rng.standard_normal(n) * 0.5
    refs = refs.astype(np.float32)
    up = rng.standard_normal(P).astype(np.float32)
    idd, off = _dev(ids, np.int32), _dev(offsets, np.int32)
    loss, ratios, stats = ls.preference_loss(dev, idd, off, ref_log_probs=_dev(refs) if ref else None, weights=_dev(w),
                                             temperature=T, **how)
    grad = _f64(ls.preference_loss_backward(dev, idd, stats, _dev(up), temperature=T))
    kw = {{"loss": "kind", "label_smoothing": "smoothing"}.get(k, k): v if isinstance(v, (str, bool)) else float(np.float32(v))
          for k, v in how.items()}
    kw.setdefault("beta", float(np.float32(0.1)))
    weights = np.ones(n) if w is None else w.astype(np.float64)
    slopes, tol_g = np.zeros(n), np.zeros(n)
    for p in range(P):
        lo, mid, hi = offsets[2 * p:2 * p + 3]
        want, s, g, slope = R.preference_pair(lp, refs.astype(np.float64) if ref else None, weights, lo, mid, hi, **kw)
        tol_s = []
        for a, b in ((lo, mid), (mid, hi)):
            on = [i for i in range(a, b) if rows[i] is not None]
            total = sum(abs(weights[i]) for i in on) if how.get("average") else 1.0
            tol_s.append(sum(abs(weights[i]) * (rows[i].tol_lp + 4 * R.EPS * (abs(lp[i]) + abs(refs[i]))) for i in on)
                         / max(total, 1e-9) + 2 * R.EPS * abs(s[len(tol_s)]))
        _near(_f64(ratios[2 * p:2 * p + 2]), s, tol_s, f"{what} ratios {p}")
        u_tol = sum(tol_s) + 2 * R.EPS * abs(s[0] - s[1])
        beta = kw["beta"]
        steep = 2 * (abs(s[0] - s[1]) + 0.5 / beta) if kw.get("kind") == "ipo" else beta
        bend = 2.0 if kw.get("kind") == "ipo" else 0.25 * beta * beta if kw.get("kind", "sigmoid") == "sigmoid" else 0.0
        # the rounding of the parts that a loss is added up from
        parts = (abs(s[0] - s[1]) + 0.5 / beta) ** 2 if kw.get("kind") == "ipo" else 2 + abs(beta * (s[0] - s[1])) + abs(kw.get("margin", 0))
        _near(float(loss[p]), want, steep * u_tol + bend * u_tol ** 2 + 8 * R.EPS * parts, f"{what} loss {p}")
        total = {k: sum(weights[i] for i in range(a, b) if rows[i] is not None) if how.get("average") else 1.0
                 for k, (a, b) in enumerate(((lo, mid), (mid, hi)))}
        for i in range(lo, hi):
            slopes[i] = g[i] * up[p]
            over = abs(weights[i] / total[i >= mid]) if total[i >= mid] else 0.0
            tol_g[i] = abs(up[p]) * over * (bend * u_tol + 8 * R.EPS * (abs(slope) + (0.5 / beta if bend == 2.0 else beta)))
    _check_gradient(grad, rows, slopes, np.zeros(n), dtype, f"{what} gradient", tol_g)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("how", [{}, {"average": True, "loss": "ipo"}, {"loss": "hinge", "beta": 0.4, "margin": 0.3},
                                 {"label_smoothing": 0.1}, {"ref": False, "average": True, "beta": 2.0, "margin": 0.5},
                                 {"loss": "ipo", "beta": 0.5}, {"loss": "hinge", "beta": 1e-3}])
def test_preference_forms(dtype, how):
    rng = np.random.default_rng(21)
    V = 1003
    for n, offsets in ((2, [0, 1, 2]), (30, [0, 7, 9, 9, 20, 20, 20, 23, 29]), (64, [3, 30, 60])):
        if len(offsets) % 2 == 0:
            offsets = offsets[:-1]
        dev, x = _logits(_normal(rng, n, V), dtype, 3, 2)
        ids = rng.integers(0, V, n)
        ids[n // 2] = -1
        w = (rng.integers(0, 4, n) / 2).astype(np.float32)
        _preference(dev, x, ids, offsets, dtype, 1.0, rng, f"{n} rows {how}", w=w, **how)
        _preference(dev, x, ids, offsets, dtype, 0.8, rng, f"{n} rows, no weights, {how}", **how)


@pytest.mark.parametrize("dtype", DTYPES)
def test_preference_batches(dtype):
    rng = np.random.default_rng(22)
    for n, V, cuts in ((900, 1000, 7), (130, 32003, 3), (1500, 77, 1)):
        offsets = [0] + sorted(rng.integers(1, n - 2, 2 * cuts - 1).tolist()) + [n - 1]
        dev, x = _logits(_normal(rng, n, V), dtype)
        _preference(dev, x, rng.integers(0, V, n), offsets, dtype, 1.0, rng, f"{n} x {V}")


def test_preference_bad_offsets():
    """Offsets that descend or leave the rows: NaN for that pair, 0 for its rows' gradients, the others as they are."""
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(23)
    dev, _ = _logits(_normal(rng, 12, 300), "f32")
    idd = _dev(rng.integers(0, 300, 12), np.int32)
    good = ls.preference_loss(dev, idd, _dev([0, 2, 4, 6, 8], np.int32))
    for bad in ([0, 2, 4, 3, 8], [0, 2, 4, 6, 13], [0, 2, 4, 20, 8], [0, 2, 4, -5, 8], [0, 2, 4, 2 ** 31 - 1, -2 ** 31],
                [0, 2, 4, 3, 3], [0, 2, 4, 4, 1]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        loss, ratios, stats = ls.preference_loss(dev, idd, _dev(bad, np.int32), error_word=err)
        assert int(err) == ls.LS_ROW_ERR_BAD_OFFSETS and torch.isnan(loss[1]) and torch.isnan(ratios[2:]).all()
        grad = ls.preference_loss_backward(dev, idd, stats)
        assert not grad[4:].any()
        if bad[-1] >= 4:  # rows 0 to 3 lie within what the list spans
            assert torch.equal(loss[0], good[0][0]) and grad[:4].any(-1).all()
        else:
            assert torch.isnan(loss[0]) and not grad.any()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for bad in ([-1, 2, 4], [5, 3, 8], [2, 9, 5]):
        loss, _, stats = ls.preference_loss(dev, idd, _dev(bad, np.int32), error_word=err)
        assert torch.isnan(loss).all() and not ls.preference_loss_backward(dev, idd, stats).any()


def test_preference_without_pairs_or_rows():
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(24)
    dev, _ = _logits(_normal(rng, 3, 50), "bf16")
    idd = _dev([1, 2, 3], np.int32)
    loss, ratios, stats = ls.preference_loss(dev, idd, _dev([0], np.int32))
    assert loss.shape == (0,) and ratios.shape == (0,) and not ls.preference_loss_backward(dev, idd, stats).any()
    loss, ratios, _ = ls.preference_loss(dev[:0], idd[:0], _dev([0, 0, 0, 0, 0], np.int32))
    assert torch.allclose(loss, torch.full((2,), float(np.log(2.0)), device="cuda"), rtol=2e-7) and not ratios.any()
    # a gradient from above that is too short is seen, not read past its end
    _, _, stats = ls.preference_loss(dev, idd, _dev([0, 1, 2, 2, 3], np.int32))
    grad = ls.preference_loss_backward(dev, idd, stats, _dev([1.0]))
    assert torch.isfinite(grad[:2]).all() and torch.isnan(grad[2]).all()
    assert torch.isnan(ls.preference_loss_backward(dev, idd, stats, _dev(np.zeros(0)))).all()


# -- gradients against differences, autograd, in place, streams, graphs ----------


@pytest.mark.parametrize("op", ["score", "policy", "preference"])
def test_gradient_against_differences(op):
    """fp32 losses are off by about 1e-6, so differences over 2^-5 are by 1e-4, and h^2 / 6 of third derivatives below 1."""
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(31)
    V, n, h = 24, 6, 2.0 ** -5
    x = _normal(rng, n, V, 1.0)
    ids = _dev(rng.integers(0, V, n), np.int32)
    g = _dev(rng.standard_normal(n))
    old = ls.token_log_probs(_dev(x), ids)[0] - _dev([0.05, -0.1, 0.6, -0.7, 0.1, 0.0])

    def total(t):
        if op == "score":
            lp, ent = ls.score(t, ids, entropy=True)
            return (g * lp).sum() + (g.flip(0) * ent).sum()
        if op == "policy":
            return (g * ls.policy(t, ids, g, old, old - 0.3, kl_coef=0.3, entropy_coef=0.2)[0]).sum()
        return ls.preference(t, ids, _dev([0, 2, 3, 4, 6], np.int32), old, beta=0.5)[0].sum()

    leaf = _dev(x).requires_grad_()
    total(leaf).backward()
    grad = leaf.grad.cpu().numpy()
    for i in range(n):
        for j in range(0, V, 5):
            d = np.zeros_like(x)
            d[i, j] = h
            up, dn = (float(total(_dev(x + s * d))) for s in (1, -1))
            assert abs((up - dn) / (2 * h) - grad[i, j]) < 1e-3, (op, i, j)


def test_autograd_parts():
    """Gradients of a sum, of one of two outputs, of expanded gradients from above, and of leaves used twice."""
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(32)
    ids = _dev(rng.integers(0, 90, 5), np.int32)
    leaf = _dev(_normal(rng, 5, 90)).requires_grad_()
    lp, h = ls.score(leaf, ids)
    assert h is None
    a, = torch.autograd.grad(lp.sum(), leaf)
    lp, h = ls.score(leaf, ids, 1.0, True)
    b, = torch.autograd.grad(lp.sum(), leaf, retain_graph=True)
    assert torch.equal(a, b)
    c, = torch.autograd.grad(h.sum(), leaf, retain_graph=True)
    both, = torch.autograd.grad(lp.sum() + h.sum(), leaf)
    assert torch.allclose(both, b + c, atol=1e-6)
    loss, metrics = ls.policy(leaf, ids, lp.detach())
    assert not metrics.requires_grad and torch.equal(metrics[:, 0], lp.detach())
    loss, ratios = ls.preference(leaf, ids, _dev([0, 2, 5], np.int32))
    assert not ratios.requires_grad
    loss.sum().backward()
    loss, _ = ls.preference(leaf, ids, _dev([0, 2, 5], np.int32))
    first = leaf.grad.clone()
    loss.backward(torch.ones(1, device="cuda").expand(1))
    assert torch.equal(leaf.grad, 2 * first)
    # leaves that need no gradient
    assert not ls.policy(leaf.detach(), ids, lp.detach())[0].requires_grad


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1001, 40000])
def test_in_place_and_strided_gradients(dtype, V):
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(33)
    n = 7
    dev, _ = _logits(_normal(rng, n, V), dtype, 3, 9)
    ids, adv = _dev(rng.integers(0, V, n), np.int32), _dev(rng.standard_normal(n))
    how = {"entropy_coef": 0.1}
    loss, grad, metrics = ls.policy_loss_grad(dev, ids, adv, **how)
    _, _, stats = ls.policy_loss(dev, ids, adv, **how)
    back = ls.policy_loss_backward(dev, ids, stats)
    buf = torch.full((n, V + 24), 5.0, dtype=dev.dtype, device="cuda")
    for f in (lambda out: ls.policy_loss_grad(dev, ids, adv, out_grad=out, **how)[1],
              lambda out: ls.policy_loss_backward(dev, ids, stats, out=out)):
        for shift in (0, 1, 16):
            buf.fill_(5.0)
            f(buf[:, shift:shift + V])
            assert torch.equal(buf[:, shift:shift + V], grad) or torch.equal(buf[:, shift:shift + V], back)
            assert (buf[:, :shift] == 5).all() and (buf[:, shift + V:] == 5).all()
    def copy():  # a row's sums are added up in an order that its alignment decides: the copy has the same
        return _logits(_f64(dev), dtype, 3, 9)[0]

    again = copy()
    assert torch.equal(ls.policy_loss_backward(again, ids, stats, out=again), back)
    again = copy()
    version = again._version
    loss3, out, metrics3 = ls.policy_loss_grad(again, ids, adv, out_grad=again, **how)
    assert out is again and again._version > version
    assert torch.equal(again, grad) and torch.equal(loss3, loss) and torch.equal(metrics3, metrics)


def test_streams_graphs_and_repetition():
    """Explicit streams, calls at the same time, captured and replayed ones: the same bits."""
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(34)
    n, V = 300, 32000
    dev, _ = _logits(_normal(rng, n, V), "bf16")
    ids, adv = _dev(rng.integers(0, V, n), np.int32), _dev(rng.standard_normal(n))
    off = _dev([0, 70, 100, 180, 290], np.int32)

    def step(x):
        lp, h, st = ls.token_log_probs(x, ids, entropy=True)
        loss, m, sp = ls.policy_loss(x, ids, adv, old_log_probs=lp, entropy_coef=0.1)
        pl, pr, sq = ls.preference_loss(x, ids, off, ref_log_probs=lp)
        return [lp, h, loss, m, pl, pr, ls.token_log_probs_backward(x, ids, st, adv, adv),
                ls.policy_loss_backward(x, ids, sp), ls.preference_loss_backward(x, ids, sq),
                *ls.policy_loss_grad(x, ids, adv, lp)]

    want = step(dev)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        out = []
        for s in (s1, s2):
            with torch.cuda.stream(s):
                out.append(step(dev))
        torch.cuda.synchronize()
        for got in out:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    lp = ls.token_log_probs(dev, ids, stream=s1)[0]
    s1.synchronize()
    assert torch.equal(lp, ls.token_log_probs(dev, ids)[0])
    x = dev.clone()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = step(x)
        graphs.append((g, held))
    x.copy_(dev.flip(0))
    other = step(x)
    for g, held in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, held in graphs:
        assert all(torch.equal(a, b) for a, b in zip(held, other))
