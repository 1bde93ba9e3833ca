"""How exact log-probs and entropies are on ordinary rows: mean and rms error
against 64 bits over many rows, from the roundings that are left.

terms  Exponents below 32 in base 2 are rounded to 2^-19, rms 2^-19 ln 2 / sqrt(12) of
       a term; the exponential itself is off by 2^-22.5 at most, rms a third of that:
       together e = 3.9e-7 of each term.  ln S is off by e sqrt(sum q^2), H by e sqrt(sum
       (q (ln q + H))^2) for the exponents and by the same with ln q + H - 1 for the
       exponential.
factor log2(e) in fp32 is short by 1.335e-8 of itself, as if T were larger: with it H
       rises by that times the variance of ln q over the row, and ln q of a token drawn
       from the row moves by that times its distance from the mean, rms the deviation.
sums   An addition is off by 2.5e-8 of its result (2^-24 / sqrt(3) of it at a power of
       two, half of that below the next, between them rms 2.5e-8).  Partial sums that are
       joined in pairs give 2 such variances in all (1 + 1/2 + 1/4 ...), a thread's chain
       of 64 over 128 threads half a one: 4e-8 of S and of E.  In H, E / S counts ln S - H.
rest   The result is rounded once, rms ulp / sqrt(12); log2 and S's sums 5e-8.

The rms over n rows is within a quarter of that (five of its standard deviations and
more).  The exponential's mean error, 5e-8 of a term, is compensated: a third of it
may be left in a mean over rows, beside the factor's part and 4 standard errors."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
E, FACTOR, SUMS = 3.9e-7, 1.335e-8, 4e-8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


def _drawn(x, dtype, gen):
    import torch
    x = x.to(torch.bfloat16) if dtype == "bf16" else x
    noise = torch.empty(x.shape, device="cuda").exponential_(generator=gen).log_()
    return x, (x.float() - noise).argmax(1)


def _step(v):
    import torch
    return 2.0 ** (torch.floor(torch.log2(v.abs())) - 23) / 12 ** 0.5


def _errors(x, ids):
    """{(what, with entropies): (errors, variances from the terms, from the rest, shifts by the factor)} of each row."""
    import logits_sampling_gb300 as ls
    import torch
    z = x.double()
    log_q = torch.log_softmax(z, 1)
    ln_s = torch.logsumexp(z, 1) - z.amax(1)
    del z
    q = log_q.exp()
    H = -(q * log_q).sum(1)
    spread = (q * (log_q + H[:, None]) ** 2).sum(1)
    lp = log_q.gather(1, ids[:, None])[:, 0]
    inner = torch.maximum((log_q + H[:, None]).abs(), (log_q + H[:, None] - 1).abs())
    terms = {"lp": E ** 2 * (q ** 2).sum(1), "H": E ** 2 * ((q * inner) ** 2).sum(1)}
    rest = {"lp": _step(lp) ** 2 + 5e-8 ** 2 + FACTOR ** 2 * spread,
            "H": _step(H) ** 2 + 5e-8 ** 2 + SUMS ** 2 * (ln_s - H) ** 2}
    shift = {"lp": torch.zeros_like(lp), "H": FACTOR * spread}
    del log_q, q, inner
    out = {}
    for entropy in (False, True):
        got, h, _ = ls.token_log_probs(x, ids.to(torch.int32), entropy=entropy)
        off = {"lp": got.double() - lp, "H": h.double() - H if entropy else None}
        for what in ("lp", "H") if entropy else ("lp",):
            out[what, entropy] = [v.cpu().numpy() for v in (off[what], terms[what], rest[what], shift[what])]
    return out


def _check(off, variance, shift, what, mean_bound):
    rms, mean, bound = np.sqrt((off ** 2).mean()), off.mean() - shift.mean(), 1.25 * np.sqrt((variance + shift ** 2).mean())
    print(f"{what}: rms {rms:.3g} (bound {bound:.3g}), mean {mean:.3g} + {shift.mean():.3g} (bound {mean_bound:.3g})")
    assert rms <= bound, (what, rms, bound)
    assert abs(mean) <= mean_bound, (what, mean, mean_bound)


@pytest.mark.parametrize("dtype,n,V", [("bf16", 1024, 32000), ("f32", 1024, 32000), ("bf16", 512, 128256),
                                       ("f32", 512, 128256)])
def test_rows_with_the_same_head(dtype, n, V):
    """Rows as a language model's are: N(0, 3) with 200 ids on a Zipf-shaped head below 20.  The head's values are the
    same in all rows, and so are their terms' errors: a mean over rows has all of the terms' error in it."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = torch.empty(n, V, device="cuda").normal_(0.0, 3.0, generator=gen)
    ids = (torch.randint(V, (n, 1), device="cuda", generator=gen)
           + torch.randint(1, V // 200, (n, 200), device="cuda", generator=gen).cumsum(1)) % V
    rank = torch.arange(1, 201, device="cuda", dtype=torch.float32)
    x.scatter_(1, ids, (20.0 - 1.1 * rank.log()).expand(n, 200))
    for (what, entropy), (off, terms, rest, shift) in _errors(*_drawn(x, dtype, gen)).items():
        mean = 4 * np.sqrt(terms.mean() + rest.mean() / n) + 5.05e-8 / 3
        _check(off, terms + rest, shift, f"{what} {dtype} {n} x {V}, entropy {entropy}", mean)


@pytest.mark.parametrize("dtype,n,V,scale", [("bf16", 8192, 16384, 1.5), ("f32", 8192, 16384, 1.5),
                                             ("bf16", 2048, 128256, 3.0), ("f32", 2048, 128256, 3.0)])
def test_rows_at_any_level(dtype, n, V, scale):
    """Rows whose maxima lie at different places: their errors are independent, and the mean shows what all have."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(n)
    x = torch.empty(n, V, device="cuda").normal_(0.0, scale, generator=gen)
    x += torch.empty(n, 1, device="cuda").uniform_(-8.0, 8.0, generator=gen)
    x, ids = _drawn(x, dtype, gen)
    parts = {}
    for at in range(0, n, 1024):
        for key, values in _errors(x[at:at + 1024], ids[at:at + 1024]).items():
            parts.setdefault(key, []).append(values)
    for (what, entropy), values in parts.items():
        off, terms, rest, shift = (np.concatenate(v) for v in zip(*values))
        mean = 4 * np.sqrt((terms + rest).mean() / n) + 5.05e-8 / 3
        _check(off, terms + rest, shift, f"{what} {dtype} {n} x {V}, entropy {entropy}", mean)
