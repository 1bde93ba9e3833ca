"""Plain definitions in 64 bits (numpy) of the operators on logits rows, one row
at a time, and the tolerances their fp32 arithmetic earns.

U is the unit roundoff of fp32.  SUM_REL bounds the relative error of a row's
sum of exponentials in fp32: chains of at most 150 additions per thread and a
tree of at most 15 levels (165 U = 1.0e-5) over terms whose own error (exponent
argument: 3 U |t|, weighed by the term; hardware base-2 exponential: 2^-22)
stays below 1e-5 in the weighted mean."""
import numpy as np

U = 2.0 ** -24
SUM_REL = 2e-5


def to_dtype(x, dtype):
    """The values that a tensor of `dtype` ("f32" or "bf16") holds, as float32."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    return t.to(torch.bfloat16).float().numpy() if dtype == "bf16" else t.numpy()


def device_matrix(x, dtype, col_off=0, pad=0):
    """x on the device as rows of a wider buffer: row stride col_off + V + pad,
    first entry col_off past an aligned address."""
    import torch
    t = torch.zeros((x.shape[0], col_off + x.shape[1] + pad), dtype=torch.float32)
    t[:, col_off:col_off + x.shape[1]] = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    if dtype == "bf16":
        t = t.to(torch.bfloat16)
    return t.cuda()[:, col_off:col_off + x.shape[1]]


def within(got, ref, tol, dtype):
    """Whether each value lies between ref - tol and ref + tol as they round to
    `dtype` (rounding keeps order, so any fp32 result within tol of ref does)."""
    import torch
    t = torch.bfloat16 if dtype == "bf16" else torch.float32

    def store(v):  # through fp32, as the kernels store
        with np.errstate(over="ignore"):
            return torch.from_numpy(np.asarray(v, np.float64).astype(np.float32)).to(t).double().numpy()

    got = np.asarray(got, np.float64)
    return (store(ref - tol) <= got) & (got <= store(ref + tol))


# -- penalties, bias, mask -------------------------------------------------------


def process_row(x, tokens=(), prompt_len=0, rho=1.0, presence=0.0, frequency=0.0, bias=None, allowed=None):
    """Returns (y float64, touched bool, tol float64 before the store's rounding)."""
    x = np.asarray(x, np.float64)
    V = len(x)
    seen = np.zeros(V, bool)
    c = np.zeros(V)
    for q, t in enumerate(tokens):
        if 0 <= t < V:
            seen[t] = True
            c[t] += q >= prompt_len
    b = np.zeros(V)
    for j, v in (bias or {}).items():
        if 0 <= j < V:
            b[j] = v
    touched = seen | (b != 0)
    with np.errstate(all="ignore"):
        y = np.where(seen, np.where(x > 0, x / rho, x * rho), x)
        size = np.abs(y)
        y = y - frequency * c - np.where(c > 0, presence, 0.0)
        y = y + b
        size = size + np.abs(frequency * c) + np.where(c > 0, abs(presence), 0.0) + np.abs(b)
    y = np.where(touched & np.isnan(y), -np.inf, y)
    if allowed is not None:
        y = np.where(allowed, y, -np.inf)
        touched = touched | ~np.asarray(allowed)
    # five roundings, none of a value larger than the sum of the parts
    tol = 5 * U * np.where(np.isfinite(size), size, 0.0)
    return y, touched, tol


def pack_mask(allowed, words=None):
    """bool [rows, V] -> int32 [rows, words], bit j % 32 of word j / 32."""
    rows, V = allowed.shape
    words = words or (V + 31) // 32
    bits = np.zeros((rows, words * 32), np.uint64)
    bits[:, :V] = allowed
    w = (bits.reshape(rows, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return w.view(np.int32)


# -- top log-probs ----------------------------------------------------------------


def guard(x):
    x = np.asarray(x, np.float64)
    return np.where(np.isnan(x), -np.inf, x)


def row_lse(x, T):
    """(max, ln sum exp((x - max) / T)) with the limit at an infinite maximum."""
    x = guard(x)
    M = x.max()
    with np.errstate(all="ignore"):
        e = np.where(x == M, 1.0, np.exp((x - M) / T))
    return M, np.log(e.sum())


def top_row(x, k, T):
    """(ids, log_probs, lse) or None for a row with nothing above -inf."""
    x = guard(x)
    M, ln_s = row_lse(x, T)
    if M == -np.inf:
        return None
    order = np.lexsort((np.arange(len(x)), -x))[:k]
    order = order[x[order] > -np.inf]
    with np.errstate(all="ignore"):
        lp = np.where(x[order] == M, 0.0, (x[order] - M) / T) - ln_s
    ids = np.full(k, -1, np.int64)
    out = np.full(k, -np.inf)
    ids[:len(order)] = order
    out[:len(order)] = lp
    return ids, out, M / T + ln_s


def top_tolerance(lp):
    """Per log-prob: the sum's error, and three roundings no larger than the value's parts."""
    return SUM_REL + 6 * U * (np.abs(lp) + 20.0)


# -- distillation -------------------------------------------------------------------


def distill_row(x, ids, log_probs, T, tail, w=1.0, g=1.0):
    """One row: (loss, tol_loss, gradient, tol_grad before the store's rounding); NaN loss and gradient for a
    row with nothing above -inf."""
    x = guard(x)
    V = len(x)
    if w == 0:
        return 0.0, 0.0, np.zeros(V), np.zeros(V)
    M, ln_s = row_lse(x, T)
    if M == -np.inf:
        return np.nan, 0.0, np.full(V, np.nan), np.zeros(V)
    t = np.asarray(log_probs, np.float64)
    ids = np.asarray(ids)
    keep = (ids >= 0) & (ids < V) & (t > -np.inf)
    ids, t = ids[keep], t[keep]
    K = max(len(ids), 1)
    with np.errstate(all="ignore"):
        log_q = np.where(x == M, 0.0, (x - M) / T) - ln_s
    q = np.exp(log_q)
    p = np.exp(t)
    P = p.sum()
    if tail == "renorm":
        p, t = (p / P, t - np.log(P)) if P > 0 else (p, t)
        A = 1.0 if P > 0 else 0.0
    else:
        A = P
    live = p > 0
    with np.errstate(all="ignore"):
        loss = (p[live] * (t[live] - log_q[ids[live]])).sum()
        size = (p[live] * (np.abs(t[live]) + np.abs(log_q[ids[live]]) + 2)).sum()
    mass_err = (K + 8) * U * 2
    tol = SUM_REL * A + 16 * U * size + mass_err * A * 2
    rest = np.ones(V, bool)
    rest[ids] = False
    d = A * q
    np.subtract.at(d, ids, p)
    tol_d = 5e-5 * A * q
    np.add.at(tol_d, ids, (2.0 ** -21 + mass_err) * p)
    tol_d += mass_err * q
    if tail == "bucket" and rest.any() and x[rest].max() > -np.inf:
        pr = max(1 - P, 0.0)
        Mr, ln_sr = row_lse(x[rest], T)
        with np.errstate(all="ignore"):
            ratio = np.where(rest, np.exp(np.where(x == Mr, 0.0, (x - Mr) / T) - ln_sr), 0.0)
            log_qr = (0.0 if Mr == M else (Mr - M) / T) + ln_sr - ln_s
        # p_r = 1 - P holds P's own absolute error; where it comes within it, p_r itself may be 0
        if pr > 0:
            loss = loss + pr * (np.log(pr) - log_qr)
        tol = tol + SUM_REL * 2 * pr + 16 * U * pr * (abs(log_qr) + abs(np.log(max(pr, U)))) \
            + 2 * mass_err * (abs(np.log(max(pr, mass_err))) + 1 + abs(log_qr))
        d = d + pr * q - pr * ratio
        tol_d = tol_d + 5e-5 * pr * (q + ratio) + mass_err * (q + ratio)
    s = w * g / T
    tiny = 1e-37 * max(abs(s), 1.0)  # exponentials below 2^-126 are flushed
    tol_d = abs(s) * tol_d + 2 * U * np.abs(s * d) + tiny
    return w * loss, abs(w) * tol + U * abs(w * loss), s * d, tol_d
