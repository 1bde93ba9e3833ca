"""The operators on sampled tokens from their definitions in 64 bits, and how far
fp32 kernels may be from them.

Tolerances, with eps = 2^-24 (half a step of fp32) and y = (x - M) / T:
  term      a term exp(y) of a row's sum: the factor log2(e) / T and the exponent
            are rounded three times (3 eps |y|), the exponential is off by at
            most 2^-22, and every time the running maximum rises (at most once
            per stage of 512 units, and twice when threads and CTAs are joined)
            the sums are multiplied by one more such factor; where a sum is made
            against a reference g below the maximum instead, it is not multiplied
            but each exponent is g larger: 3 eps g, which is below the 2^-22 (stages
            + 4) of those factors for g up to 5
  sum       added up by a thread over its entries, then over the threads: one
            rounding per addition of a thread, and 16 more
  ln S      relative error of S, and its own two roundings
  lp        y of the token (2 eps |y|), ln S, and the subtraction
  H         ln S, and sum q |y| with each term's error
  q_j       its own term's error, S's, and a product's rounding
A gradient is rounded once to its type; a term below 2^-126 may be 0."""
import numpy as np

EPS = 2.0 ** -24
EXP = 2.0 ** -22
TINY = 2.0 ** -120
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


class Row:
    """lp, H, q of one row (x: float64 values of the logits; token: its id)."""

    def __init__(self, x, token, T, entry_bytes=4):
        x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))
        self.T, self.token, self.V = T, token, len(x)
        self.M = x.max()
        with np.errstate(invalid="ignore"):
            y = np.where(x == self.M, 0.0, (x - self.M) / T)
        e = np.exp(y)
        self.S = e.sum()
        self.q = e / self.S
        self.some = self.M > -np.inf
        if not self.some:
            self.lp = self.H = np.nan
            self.q = np.full(self.V, np.nan)
            return
        self.log_q = y - np.log(self.S)
        self.lp = self.log_q[token]
        live = self.q > 0
        self.H = -(self.q[live] * self.log_q[live]).sum()
        # tolerances
        units = self.V * entry_bytes / 32 + 2
        stages = np.ceil(units / 512)
        self.ay = np.where(live, np.abs(np.where(live, y, 0.0)), 0.0)
        term = 3 * EPS * self.ay + EXP * (stages + 4)
        adds = (self.V / 256 + 32 + 16) * EPS
        self.term = term
        self.tol_S = (self.q * term).sum() + adds
        lnS = np.log(self.S)
        self.tol_lnS = self.tol_S + 2 * EPS * lnS + EPS
        a = abs(y[token]) if np.isfinite(y[token]) else 0.0
        self.tol_lp = 2 * EPS * a + self.tol_lnS + EPS * (abs(self.lp) if np.isfinite(self.lp) else 0.0)
        self.tol_H = self.tol_lnS + (self.q * self.ay * (term + adds + self.tol_S + 4 * EPS)).sum() + EPS * abs(self.H)

    def gradient(self, g_lp, g_H=0.0):
        """d/dx of g_lp lp + g_H H, and its tolerance before rounding to the logits' type."""
        if not self.some:
            return np.full(self.V, np.nan), np.zeros(self.V)
        log_q = np.where(self.q > 0, self.log_q, 0.0)
        inner = g_lp + g_H * (log_q + self.H)
        d = -self.q * inner
        d[self.token] += g_lp
        tol_q = self.term + self.tol_S + 4 * EPS
        tol_inner = 3 * EPS * (abs(g_lp) + abs(g_H) * (np.abs(log_q) + abs(self.H) + np.log(self.S))) \
            + abs(g_H) * (3 * EPS * self.ay + self.tol_lnS + self.tol_H)
        tol = self.q * (np.abs(inner) * tol_q + tol_inner)
        tol[self.token] += abs(g_lp) * (self.q[self.token] * (self.tol_lp + 4 * EPS) + 4 * EPS * (1 - self.q[self.token]))
        # a term below 2^-126 of the largest counts 0 (S >= 1)
        tol += 2.0 ** -126 * (abs(g_lp) + abs(g_H) * (np.abs(log_q) + abs(self.H)))
        return d / self.T, tol / self.T + 2 * EPS * np.abs(d / self.T)


def log_ratio(a, b):
    return 0.0 if a == b == -np.inf else a - b


def kl_of(kind, d):
    """The estimate and its slope in lp."""
    if kind == "k1":
        return -d, 1.0
    if kind == "k2":
        return d * d / 2, -d
    return (np.inf if d == np.inf else np.expm1(d) - d), -np.expm1(d)


def policy_row(row, A, old=None, ref=None, w=1.0, lo=0.2, hi=0.2, dual=0.0, beta=0.0, kl="k3", eta=0.0):
    """(loss, (lp, H, kl, ratio), g_lp, g_H, tolerances of loss, of kl, of ratio and of g_lp)."""
    with np.errstate(over="ignore", invalid="ignore"):
        r = 1.0 if old is None else np.exp(log_ratio(row.lp, old))
        if not row.some:
            r = np.nan
        s = slope = 0.0
        if A != 0:
            u, v = r * A, min(max(r, 1 - lo), 1 + hi) * A
            s, slope = (u, -u) if u <= v or u != u else (v, 0.0)
            if A < 0 and dual > 0 and s < dual * A:
                s, slope = dual * A, 0.0
        k, k_slope = (0.0, 0.0) if ref is None else kl_of(kl, log_ratio(ref, row.lp))
        loss = -s + (beta * k if beta else 0.0) - (eta * row.H if eta else 0.0)
        g_lp = slope + (beta * k_slope if beta else 0.0)
    if not row.some:
        loss = g_lp = np.nan
        return w * loss, (np.nan,) * 4, g_lp, -w * eta, 0, 0, 0, 0
    d = 0.0 if ref is None else abs(log_ratio(ref, row.lp))
    l = 0.0 if old is None else abs(log_ratio(row.lp, old))
    fin = lambda v: v if np.isfinite(v) else 0.0  # noqa: E731
    tol_r = fin(r) * (row.tol_lp + EPS * fin(l) + 4 * EPS) if old is not None else 0.0
    tol_d = row.tol_lp + EPS * fin(d)
    tol_k_slope = {"k1": 0.0, "k2": tol_d, "k3": fin(np.exp(min(d, 80.0))) * (tol_d + 4 * EPS)}[kl] if ref is not None else 0.0
    tol_k = 0.0 if ref is None else fin(abs(k_slope)) * tol_d + tol_d ** 2 + 4 * EPS * (fin(abs(k)) + fin(abs(k_slope)) + fin(d))
    tol_s = abs(A) * tol_r + 4 * EPS * fin(abs(s))
    tol_loss = tol_s + abs(beta) * tol_k + abs(eta) * row.tol_H + 4 * EPS * (
        fin(abs(s)) + abs(beta) * fin(abs(k)) + abs(eta) * row.H)
    tol_g = abs(A) * tol_r * (slope != 0) + abs(beta) * tol_k_slope + 4 * EPS * (fin(abs(slope)) + abs(beta) * fin(abs(k_slope)))
    return (w * loss, (row.lp, row.H, k, r), w * g_lp, -w * eta, abs(w) * tol_loss, tol_k, tol_r, abs(w) * tol_g)


def preference_pair(lp, ref, w, lo, mid, hi, beta=0.1, kind="sigmoid", smoothing=0.0, margin=0.0, average=False):
    """(loss, s of the chosen and of the rejected answer, each row's slope {row: g}); lp None: the row does not count."""
    s, total = [], []
    for a, b in ((lo, mid), (mid, hi)):
        rows = [i for i in range(a, b) if lp[i] is not None]
        total.append(sum(w[i] for i in rows) if average else 1.0)
        v = sum(w[i] * log_ratio(lp[i], ref[i] if ref is not None else 0.0) for i in rows)
        s.append(v if not average else v / total[-1] if total[-1] else 0.0)
    with np.errstate(over="ignore", invalid="ignore"):
        u = s[0] - s[1]
        h = beta * u - margin
        if kind == "sigmoid":
            sp = lambda v: np.logaddexp(0.0, v)  # noqa: E731
            sg = lambda v: 1 / (1 + np.exp(-v))  # noqa: E731
            loss = (1 - smoothing) * sp(-h) + (smoothing * sp(h) if smoothing else 0.0)
            slope = beta * (smoothing * sg(h) - (1 - smoothing) * sg(-h))
        elif kind == "hinge":
            loss, slope = max(0.0, 1 - h), -beta if h < 1 else 0.0
        else:
            loss, slope = (u - 0.5 / beta) ** 2, 2 * (u - 0.5 / beta)
    g = {}
    for i in range(lo, hi):
        k = 0 if i < mid else 1
        g[i] = 0.0 if lp[i] is None else (1 - 2 * k) * slope * w[i] / total[k]
    return loss, s, g, slope
