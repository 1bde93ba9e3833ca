"""Timed cases of the operators that train on sampled tokens: log-probs and
entropies of given tokens, the clipped policy loss with a KL term, and the
preference loss of pairs of answers, with their gradients.

`run` computes a case in plain torch operations in 32 bits, or, with `own` set,
through the package's calls; `exact` computes the same outputs from the
definitions in 64 bits.  Rows, vocabularies and types follow the package's
serving configurations (4 x 1000, 64 x 32000, 256 x 128256, 672 x 151936 and
1024 x 262144); logits are N(0, 3) with a Zipf-shaped head, as a language
model's rows are, and the tokens are drawn from them.
"""
import math

import torch

own = False

ALPHA = (0.2, 0.28)  # how far a ratio may go below and above 1
DUAL = 3.0
BETA = 0.1


def listed():
    return [
        # one sampled token scored on its own: the call's latency
        {"name": "score 1 token", "op": "score", "dtype": "bf16", "rows": 1, "vocab": 32000, "temperature": 1.0,
         "entropy": False, "way": "loss"},
        # the rollouts of a speculative batch under the reference model: log-probs alone
        {"name": "score rollouts", "op": "score", "dtype": "bf16", "rows": 672, "vocab": 151936, "temperature": 1.0,
         "entropy": False, "way": "loss"},
        # a loss of the user's own on log-probs and entropies, an odd vocabulary: forward, then backward
        {"name": "score step odd", "op": "score", "dtype": "bf16", "rows": 333, "vocab": 32003, "temperature": 0.7,
         "entropy": True, "way": "step"},
        # the largest batch under the sampling policy, fp32 logits, with entropies: memory bandwidth
        {"name": "score large fp32", "op": "score", "dtype": "f32", "rows": 1024, "vocab": 262144, "temperature": 1.0,
         "entropy": True, "way": "loss"},
        # a training step on a few short rows: latency of forward and backward
        {"name": "policy step tiny", "op": "policy", "dtype": "f32", "rows": 8, "vocab": 1001, "temperature": 1.0,
         "kl": "k3", "entropy": True, "way": "step"},
        # one rollout's answer, loss and gradient from one call
        {"name": "policy fused small", "op": "policy", "dtype": "bf16", "rows": 64, "vocab": 32000, "temperature": 1.0,
         "kl": "k3", "entropy": False, "way": "fused"},
        # a training step whose gradient of the loss arrives from above, entropy bonus: forward, then backward
        {"name": "policy step", "op": "policy", "dtype": "bf16", "rows": 2048, "vocab": 128256, "temperature": 1.0,
         "kl": "k3", "entropy": True, "way": "step"},
        # the same batch, loss and gradient from one call
        {"name": "policy fused", "op": "policy", "dtype": "bf16", "rows": 2048, "vocab": 128256, "temperature": 1.0,
         "kl": "k2", "entropy": False, "way": "fused"},
        # the largest batch, fp32 logits
        {"name": "policy fused large fp32", "op": "policy", "dtype": "f32", "rows": 1024, "vocab": 262144,
         "temperature": 0.7, "kl": "k3", "entropy": True, "way": "fused"},
        # one pair of short answers: latency of forward and backward
        {"name": "preference step tiny", "op": "preference", "dtype": "bf16", "rows": 24, "vocab": 32000, "pairs": 1,
         "temperature": 1.0, "loss": "sigmoid", "average": False, "way": "step"},
        # a training batch of ragged pairs, padded behind the last one
        {"name": "preference step", "op": "preference", "dtype": "bf16", "rows": 2048, "vocab": 128256, "pairs": 16,
         "temperature": 1.0, "loss": "sigmoid", "average": False, "way": "step"},
        # validation on long answers, averaged over their lengths: the loss alone
        {"name": "preference loss fp32", "op": "preference", "dtype": "f32", "rows": 1024, "vocab": 151936, "pairs": 4,
         "temperature": 1.0, "loss": "ipo", "average": True, "way": "loss"},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("score", "policy", "preference"))
    vocab = log_int(1000, 262144)
    if rng.random() < 0.5:
        vocab = max(1000, vocab // 64 * 64)
    rows = min(log_int(1, 2048), (1 << 27) // vocab)
    case = {"op": op, "dtype": rng.choice(("bf16", "f32")), "rows": rows, "vocab": vocab,
            "temperature": rng.choice((0.7, 1.0, 1.3))}
    if op == "score":
        return {**case, "entropy": rng.random() < 0.5, "way": rng.choice(("loss", "step"))}
    if op == "policy":
        return {**case, "kl": rng.choice(("k1", "k2", "k3")), "entropy": rng.random() < 0.5,
                "way": rng.choice(("loss", "step", "fused"))}
    return {**case, "pairs": min(log_int(1, 64), max(1, rows // 4)), "loss": rng.choice(("sigmoid", "hinge", "ipo")),
            "average": rng.random() < 0.5, "way": rng.choice(("loss", "step"))}


# -- the layout of a batch ------------------------------------------------------


def _lengths(case):
    """Rows of each answer, chosen and rejected in turn: ragged, with a sixteenth of the batch left as padding."""
    room, answers = case["rows"] * 15 // 16, 2 * case["pairs"]
    share = [1 + 5 * s % 7 for s in range(answers)]
    return [room * k // sum(share) for k in share]


def _counted(case):
    """Which rows count: the first quarter of each text is its prompt."""
    if case["op"] == "score":
        return [True] * case["rows"]
    if case["op"] == "policy":  # rollouts of 64 rows each (in a short batch: of all its rows)
        text = min(64, case["rows"])
        return [i % text >= text // 4 for i in range(case["rows"])]
    rows = [i >= n // 4 for n in _lengths(case) for i in range(n)]
    return rows + [False] * (case["rows"] - len(rows))


# -- inputs -------------------------------------------------------------------


def _logits(case, gen):
    """N(0, 3) with 200 ids of each row (fewer in a short row) on a Zipf-shaped head below 20."""
    rows, vocab = case["rows"], case["vocab"]
    x = torch.empty(rows, vocab, device="cuda").normal_(0.0, 3.0, generator=gen)
    heads = min(200, vocab // 8)
    ids = (torch.randint(vocab, (rows, 1), device="cuda", generator=gen)
           + torch.randint(1, vocab // heads, (rows, heads), device="cuda", generator=gen).cumsum(1)) % vocab
    rank = torch.arange(1, heads + 1, device="cuda", dtype=torch.float32)
    x.scatter_(1, ids, (20.0 - 1.1 * rank.log()).expand(rows, heads))  # ids distinct: steps of 1 or more, no full turn
    return x.to(torch.bfloat16) if case["dtype"] == "bf16" else x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rows, dev = case["rows"], {"device": "cuda"}
    x = _logits(case, gen)
    z = x.float() / case["temperature"]
    noise = torch.empty_like(z).exponential_(generator=gen).log_()
    ids = (z - noise).argmax(1)  # drawn from the softmax
    lp = z.gather(1, ids[:, None])[:, 0] - z.logsumexp(1)
    del z, noise
    state = {"case": case, "logits": x, "ids": ids.to(torch.int32),
             "weights": torch.tensor(_counted(case), **dev).float()}
    if case["op"] == "score":
        state["grad_lp"] = torch.empty(rows, **dev).normal_(generator=gen) / rows
        state["grad_entropy"] = torch.empty(rows, **dev).normal_(generator=gen) / rows
        return state
    state["ref"] = lp + torch.empty(rows, **dev).normal_(0.0, 0.3, generator=gen)
    if case["op"] == "policy":
        state["weights"] /= state["weights"].sum()
        state["advantages"] = torch.empty(rows, **dev).normal_(generator=gen)
        # some updates after the rollout: ratios that are clipped on both sides, none within 1e-3 of a border, where the
        # loss's slope jumps
        d = torch.empty(rows, **dev).normal_(0.0, 0.4, generator=gen)
        for border in (1 - ALPHA[0], 1 + ALPHA[1], DUAL):
            d = torch.where((d - math.log(border)).abs() < 1e-3, math.log(border) + 2e-3, d)
        state["old"] = lp - d
        state["grad_loss"] = torch.rand(rows, generator=gen, **dev) + 0.5
        return state
    state["offsets"] = torch.tensor([0] + _lengths(case), **dev).cumsum(0).to(torch.int32)
    state["grad_loss"] = (torch.rand(case["pairs"], generator=gen, **dev) + 0.5) / case["pairs"]
    return state


# -- the calls of the package ---------------------------------------------------


def _own_score(state):
    import logits_sampling_gb300 as ls
    case, x, ids = state["case"], state["logits"], state["ids"]
    lp, entropy, stats = ls.token_log_probs(x, ids, temperature=case["temperature"], entropy=case["entropy"])
    out = [lp, entropy] if case["entropy"] else [lp]
    if case["way"] == "step":
        out.append(ls.token_log_probs_backward(
            x, ids, stats, grad_log_probs=state["grad_lp"], grad_entropy=state["grad_entropy"] if case["entropy"] else None,
            temperature=case["temperature"]))
    return out


def _own_policy(state):
    import logits_sampling_gb300 as ls
    case, x, ids = state["case"], state["logits"], state["ids"]
    how = {"old_log_probs": state["old"], "ref_log_probs": state["ref"], "weights": state["weights"],
           "temperature": case["temperature"], "clip_low": ALPHA[0], "clip_high": ALPHA[1], "dual_clip": DUAL,
           "kl_coef": 0.05, "kl": case["kl"], "entropy_coef": 0.01 if case["entropy"] else 0.0}
    if case["way"] == "fused":
        loss, grad, metrics = ls.policy_loss_grad(x, ids, state["advantages"], **how)
        return [loss, metrics, grad]
    loss, metrics, stats = ls.policy_loss(x, ids, state["advantages"], **how)
    if case["way"] == "loss":
        return [loss, metrics]
    grad = ls.policy_loss_backward(x, ids, stats, grad_loss=state["grad_loss"], temperature=case["temperature"])
    return [loss, metrics, grad]


def _own_preference(state):
    import logits_sampling_gb300 as ls
    case, x, ids = state["case"], state["logits"], state["ids"]
    loss, ratios, stats = ls.preference_loss(x, ids, state["offsets"], ref_log_probs=state["ref"],
                                             weights=state["weights"], temperature=case["temperature"], beta=BETA,
                                             loss=case["loss"], average=case["average"])
    if case["way"] == "loss":
        return [loss, ratios]
    return [loss, ratios, ls.preference_loss_backward(x, ids, stats, state["grad_loss"],
                                                      temperature=case["temperature"])]


# -- the plain forms ------------------------------------------------------------


def _softmax(state, entropy):
    """Log-probs of the tokens, entropies, and what the gradient needs of each row."""
    z = state["logits"].float() / state["case"]["temperature"]
    m = z.amax(1, keepdim=True)
    y = z - m
    e = y.exp()
    s = e.sum(1, keepdim=True)
    log_q = y - s.log()
    lp = log_q.gather(1, state["ids"].long()[:, None])[:, 0]
    h = (s.log() - (e * y).sum(1, keepdim=True) / s)[:, 0] if entropy else None
    return lp, h, log_q


def _gradient(state, log_q, h, g_lp, g_h):
    """d/dx of sum g_lp lp + g_h H."""
    inner = g_lp[:, None] if g_h is None else g_lp[:, None] + g_h[:, None] * (log_q + h[:, None])
    d = -log_q.exp() * inner
    d.scatter_add_(1, state["ids"].long()[:, None], g_lp[:, None])
    return (d / state["case"]["temperature"]).to(state["logits"].dtype)


def _plain_score(state):
    case = state["case"]
    lp, h, log_q = _softmax(state, case["entropy"])
    out = [lp, h] if case["entropy"] else [lp]
    if case["way"] == "step":
        out.append(_gradient(state, log_q, h, state["grad_lp"], state["grad_entropy"] if case["entropy"] else None))
    return out


def _plain_policy(state):
    case, a, w = state["case"], state["advantages"], state["weights"]
    lp, h, log_q = _softmax(state, case["entropy"])
    r = (lp - state["old"]).exp()
    u, v = r * a, r.clamp(1 - ALPHA[0], 1 + ALPHA[1]) * a
    s = torch.minimum(u, v)
    dual = (a < 0) & (s < DUAL * a)
    s = torch.where(dual, DUAL * a, s)
    g = torch.where((u <= v) & ~dual, -a * r, 0.0)
    d = state["ref"] - lp
    kl, slope = {"k1": (-d, torch.ones_like(d)), "k2": (d * d / 2, -d), "k3": (d.expm1() - d, -d.expm1())}[case["kl"]]
    loss = -s + 0.05 * kl
    if case["entropy"]:
        loss = loss - 0.01 * h
    counted = w != 0
    loss = torch.where(counted, w * loss, 0.0)
    columns = [lp, h if case["entropy"] else torch.zeros_like(lp), kl, r]
    metrics = torch.where(counted[:, None], torch.stack(columns, 1), 0.0)
    if case["way"] == "loss":
        return [loss, metrics]
    up = w * state["grad_loss"] if case["way"] == "step" else w
    grad = _gradient(state, log_q, h, up * (g + 0.05 * slope), up * -0.01 if case["entropy"] else None)
    return [loss, metrics, grad]


def _plain_preference(state):
    case, w, offsets = state["case"], state["weights"], state["offsets"].long()
    rows, pairs = case["rows"], case["pairs"]
    lp, _, log_q = _softmax(state, False)

    def sums(v):  # of each answer's rows
        c = torch.nn.functional.pad(v.double().cumsum(0), (1, 0))
        return (c[offsets[1:]] - c[offsets[:-1]]).float()

    count = torch.ones(2 * pairs, device="cuda")
    if case["average"]:  # over the weights' sum; an answer without rows has ratio 0
        count = torch.where(sums(w) > 0, sums(w), 1.0)
    ratios = sums(w * (lp - state["ref"])) / count
    u = ratios[0::2] - ratios[1::2]
    if case["loss"] == "sigmoid":
        hh = BETA * u
        loss, slope = torch.clamp(-hh, min=0) + (-hh.abs()).exp().log1p(), -BETA * torch.sigmoid(-hh)
    elif case["loss"] == "hinge":
        loss, slope = (1 - BETA * u).clamp(min=0), torch.where(BETA * u < 1, -BETA, 0.0)
    else:
        loss, slope = (u - 0.5 / BETA) ** 2, 2 * (u - 0.5 / BETA)
    if case["way"] == "loss":
        return [loss, ratios]
    g = torch.stack([slope, -slope], 1) * state["grad_loss"][:, None] / count.view(pairs, 2)
    row = torch.arange(rows, device="cuda")
    answer = torch.searchsorted(offsets, row, right=True) - 1
    inside = answer < 2 * pairs
    g_lp = torch.where(inside, g.reshape(-1)[answer.clamp(max=2 * pairs - 1)] * w, 0.0)
    return [loss, ratios, _gradient(state, log_q, None, g_lp, None)]


def run(state):
    if own:
        return {"score": _own_score, "policy": _own_policy, "preference": _own_preference}[state["case"]["op"]](state)
    return {"score": _plain_score, "policy": _plain_policy, "preference": _plain_preference}[state["case"]["op"]](state)


# -- the work that a pass cannot do without ---------------------------------------


def work(case):
    rows, vocab, size = case["rows"], case["vocab"], 2 if case["dtype"] == "bf16" else 4
    active = sum(_counted(case))  # a row that does not count is not read
    small = rows * {"score": 8, "policy": 40, "preference": 12}[case["op"]]
    per_entry = 5 if case.get("entropy") else 3
    if case["way"] == "loss":
        return {"bytes": active * vocab * size + small, "flops": per_entry * active * vocab}
    return {"bytes": (active + rows) * vocab * size + small, "flops": 2 * per_entry * active * vocab}


# -- the definitions in 64 bits -----------------------------------------------------


def _row_terms(s, case, i):
    """ln q of row i in 64 bits."""
    return torch.log_softmax(s["logits"][i].double() / case["temperature"], 0)


def _row_gradient(case, log_q, token, g_lp, g_h):
    q = log_q.exp()
    d = -q * g_lp
    d[token] += g_lp
    if g_h:
        h = -(q * log_q).sum()
        d -= g_h * q * (log_q + h)
    d /= case["temperature"]
    return d.to(torch.float32) if case["dtype"] == "bf16" and case["rows"] * case["vocab"] > 1 << 26 else d


def _exact_score(s, case):
    lps, hs, grads = [], [], []
    g_lp, g_h = s["grad_lp"].tolist(), s["grad_entropy"].tolist()
    for i, token in enumerate(s["ids"].tolist()):
        log_q = _row_terms(s, case, i)
        lps.append(log_q[token])
        hs.append(-(log_q.exp() * log_q).sum())
        if case["way"] == "step":
            grads.append(_row_gradient(case, log_q, token, g_lp[i], g_h[i] if case["entropy"] else 0.0))
    out = [torch.stack(lps)] + ([torch.stack(hs)] if case["entropy"] else [])
    return out + ([torch.stack(grads)] if grads else [])


def _exact_policy(s, case):
    eta = 0.01 if case["entropy"] else 0.0
    ids, w = s["ids"].tolist(), s["weights"].double().tolist()
    adv, old, ref = (s[k].double().tolist() for k in ("advantages", "old", "ref"))
    up = s["grad_loss"].double().tolist() if case["way"] == "step" else [1.0] * case["rows"]
    losses, metrics, grads = [], [], []
    for i, token in enumerate(ids):
        if w[i] == 0.0:
            losses.append(0.0)
            metrics.append([0.0] * 4)
            if case["way"] != "loss":
                kind = torch.float32 if case["dtype"] == "bf16" and case["rows"] * case["vocab"] > 1 << 26 else torch.float64
                grads.append(torch.zeros(case["vocab"], dtype=kind, device="cuda"))
            continue
        log_q = _row_terms(s, case, i)
        lp = float(log_q[token])
        h = float(-(log_q.exp() * log_q).sum()) if eta else 0.0
        ratio = math.exp(lp - old[i])
        a = adv[i]
        # the bound on a gain is the clipped ratio, on a loss DUAL
        if a >= 0:
            clipped = ratio > 1 + ALPHA[1]
            gain = a * min(ratio, 1 + ALPHA[1])
        else:
            clipped = ratio < 1 - ALPHA[0] or ratio > DUAL
            gain = a * min(max(ratio, 1 - ALPHA[0]), DUAL)
        g = 0.0 if clipped else -a * ratio
        x = math.exp(ref[i] - lp)
        if case["kl"] == "k1":
            kl, slope = lp - ref[i], 1.0
        elif case["kl"] == "k2":
            kl, slope = 0.5 * (lp - ref[i]) ** 2, lp - ref[i]
        else:
            kl, slope = x - 1.0 - (ref[i] - lp), 1.0 - x
        losses.append(w[i] * (-gain + 0.05 * kl - eta * h))
        metrics.append([lp, h, kl, ratio])
        if case["way"] != "loss":
            grads.append(_row_gradient(case, log_q, token, up[i] * w[i] * (g + 0.05 * slope), -up[i] * w[i] * eta))
    out = [torch.tensor(losses, dtype=torch.float64), torch.tensor(metrics, dtype=torch.float64)]
    return out + ([torch.stack(grads)] if grads else [])


def _exact_preference(s, case):
    ids, w, ref = s["ids"].tolist(), s["weights"].tolist(), s["ref"].double().tolist()
    up, at = s["grad_loss"].double().tolist(), s["offsets"].tolist()
    lp = [float(_row_terms(s, case, i)[t]) if w[i] else 0.0 for i, t in enumerate(ids)]
    ratios, parts = [], []
    for lo, hi in zip(at, at[1:]):
        n = math.fsum(w[lo:hi]) or 1.0 if case["average"] else 1.0
        ratios.append(math.fsum(w[i] * (lp[i] - ref[i]) for i in range(lo, hi)) / n)
        parts.append(n)
    losses, g = [], [0.0] * case["rows"]
    for p in range(case["pairs"]):
        u = ratios[2 * p] - ratios[2 * p + 1]
        if case["loss"] == "sigmoid":
            loss, slope = math.log1p(math.exp(-BETA * u)), -BETA / (1 + math.exp(BETA * u))
        elif case["loss"] == "hinge":
            loss, slope = max(0.0, 1 - BETA * u), -BETA if BETA * u < 1 else 0.0
        else:
            loss, slope = (u - 1 / (2 * BETA)) ** 2, 2 * (u - 1 / (2 * BETA))
        losses.append(loss)
        for answer, sign in ((2 * p, 1), (2 * p + 1, -1)):
            for i in range(at[answer], at[answer + 1]):
                g[i] = sign * slope * up[p] * w[i] / parts[answer]
    out = [torch.tensor(losses, dtype=torch.float64), torch.tensor(ratios, dtype=torch.float64)]
    if case["way"] == "loss":
        return out
    return out + [torch.stack([_row_gradient(case, _row_terms(s, case, i), t, g[i], 0.0) for i, t in enumerate(ids)])]


def exact(case, seed):
    state = prepare(case, seed)
    return {"score": _exact_score, "policy": _exact_policy, "preference": _exact_preference}[case["op"]](state, case)
