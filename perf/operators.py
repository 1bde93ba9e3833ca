"""Timed cases of the operators on logits rows: penalties, biases and grammar
masks; the top log-probs of a row; the distillation loss from a teacher's top
log-probs, with its gradient.

`run` computes a case in plain torch operations in 32 bits, or, with `own` set,
through the package's calls; `exact` computes the same outputs from the
definitions in 64 bits.  Rows, vocabularies and types follow the package's
serving configurations (4 x 1000, 64 x 32000, 256 x 128256, 672 x 151936 and
1024 x 262144); logits are N(0, 3) with a Zipf-shaped head, as a language
model's rows are.
"""
import math

import torch

own = False

KINDS = ("process", "top", "distill")
TAILS = ("drop", "renorm", "bucket")


def listed():
    return [
        # one request decoding on its own: the call's latency
        {"name": "penalties 1 request", "op": "process", "dtype": "bf16", "rows": 1, "vocab": 32000, "history": 256,
         "per_request": 1, "bias": 0, "mask": False, "gather": False},
        # a small decode batch, an odd vocabulary: rows start at every alignment
        {"name": "penalties decode odd", "op": "process", "dtype": "bf16", "rows": 63, "vocab": 32003, "history": 2048,
         "per_request": 1, "bias": 32, "mask": True, "gather": False},
        # a full serving batch with long conversations, some rows under a grammar
        {"name": "penalties batch", "op": "process", "dtype": "bf16", "rows": 256, "vocab": 128256, "history": 8192,
         "per_request": 1, "bias": 16, "mask": True, "gather": False},
        # the largest batch, fp32 logits: memory bandwidth
        {"name": "penalties large fp32", "op": "process", "dtype": "f32", "rows": 1024, "vocab": 262144, "history": 2048,
         "per_request": 1, "bias": 16, "mask": True, "gather": False},
        # a few short rows, the five best: latency
        {"name": "top 5 tiny", "op": "top", "dtype": "f32", "rows": 4, "vocab": 1000, "k": 5, "temperature": 1.0,
         "gather": False},
        # what a serving API returns beside each sampled token of a decode batch
        {"name": "top 20 decode", "op": "top", "dtype": "bf16", "rows": 64, "vocab": 32000, "k": 20, "temperature": 1.0,
         "gather": False},
        # the same for the verified rows of a speculative batch, gathered out of a larger buffer
        {"name": "top 20 speculative", "op": "top", "dtype": "bf16", "rows": 672, "vocab": 151936, "k": 20,
         "temperature": 1.0, "gather": True},
        # a teacher scoring a batch of training positions
        {"name": "top 64 teacher", "op": "top", "dtype": "bf16", "rows": 2048, "vocab": 128256, "k": 64,
         "temperature": 2.0, "gather": False},
        # a training step on a few short rows: latency of forward and backward
        {"name": "distill step tiny", "op": "distill", "dtype": "f32", "rows": 8, "vocab": 1001, "k": 8,
         "temperature": 2.0, "tail": "bucket", "way": "step"},
        # validation: the loss alone
        {"name": "distill loss", "op": "distill", "dtype": "bf16", "rows": 672, "vocab": 151936, "k": 20,
         "temperature": 1.0, "tail": "drop", "way": "loss"},
        # a training step whose gradient of the loss arrives from the layers above: forward, then backward
        {"name": "distill step", "op": "distill", "dtype": "bf16", "rows": 2048, "vocab": 128256, "k": 64,
         "temperature": 2.0, "tail": "bucket", "way": "step"},
        # the largest training batch, loss and gradient from one call, fp32 logits
        {"name": "distill fused large fp32", "op": "distill", "dtype": "f32", "rows": 1024, "vocab": 262144, "k": 128,
         "temperature": 1.0, "tail": "renorm", "way": "fused"},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(KINDS)
    dtype = rng.choice(("bf16", "f32"))
    vocab = log_int(1000, 262144)
    if rng.random() < 0.5:
        vocab = max(1000, vocab // 64 * 64)
    rows = min(log_int(1, 2048), (1 << 28) // vocab)
    if op == "process":
        return {"op": op, "dtype": dtype, "rows": min(rows, 1024), "vocab": vocab, "history": log_int(16, 8192),
                "per_request": rng.choice((1, 1, 4, 5)), "bias": rng.choice((0, 1, 16, 300)),
                "mask": rng.random() < 0.5, "gather": rng.random() < 0.25}
    k = log_int(1, 256)
    if op == "top":
        return {"op": op, "dtype": dtype, "rows": rows, "vocab": vocab, "k": k,
                "temperature": rng.choice((0.5, 1.0, 2.0)), "gather": rng.random() < 0.25}
    return {"op": op, "dtype": dtype, "rows": min(rows, (1 << 27) // vocab * 2), "vocab": vocab, "k": k,
            "temperature": rng.choice((0.5, 1.0, 2.0)), "tail": rng.choice(TAILS),
            "way": rng.choice(("loss", "step", "fused"))}


# -- inputs -------------------------------------------------------------------


def _logits(case, rows, gen):
    """N(0, 3) with 200 ids of each row (fewer in a short row) on a Zipf-shaped head below 20."""
    vocab = case["vocab"]
    x = torch.empty(rows, vocab, device="cuda").normal_(0.0, 3.0, generator=gen)
    heads = min(200, vocab // 8)
    ids = (torch.randint(vocab, (rows, 1), device="cuda", generator=gen)
           + torch.randint(1, vocab // heads, (rows, heads), device="cuda", generator=gen).cumsum(1)) % vocab
    rank = torch.arange(1, heads + 1, device="cuda", dtype=torch.float32)
    x.scatter_(1, ids, (20.0 - 1.1 * rank.log()).expand(rows, heads))  # ids distinct: steps of 1 or more, no full turn
    return x.to(torch.bfloat16) if case["dtype"] == "bf16" else x


def _source(case, rows, gen):
    """The logits buffer, and the rows of it that a case takes (None: all, in order)."""
    if not case["gather"]:
        return _logits(case, rows, gen), None
    buf = rows + rows // 2 + 1
    gather = torch.randperm(buf, device="cuda", generator=gen)[:rows].to(torch.int32)
    return _logits(case, buf, gen), gather


def _process_state(case, gen):
    rows, vocab, per = case["rows"], case["vocab"], case["per_request"]
    requests = -(-rows // per)
    logits, gather = _source(case, rows, gen)
    dev = {"device": "cuda"}
    cap = case["history"]
    # text repeats itself: ids of a history crowd towards the low end of a per-request window
    u = torch.rand(requests, cap, generator=gen, **dev)
    base = torch.randint(vocab, (requests, 1), generator=gen, **dev)
    tokens = ((base + (u.pow(3) * vocab).long()) % vocab).to(torch.int32)
    longest = torch.rand(requests, generator=gen, **dev)
    seq = (16 * (cap / 16) ** longest).to(torch.int32).clamp(1, cap)
    prompt = (seq * torch.rand(requests, generator=gen, **dev)).to(torch.int32)
    state = {
        "logits": logits, "gather": gather, "tokens": tokens, "seq_lens": seq, "prompt_lens": prompt,
        "repetition": 1.0 + 0.5 * torch.rand(requests, generator=gen, **dev),
        "presence": torch.rand(requests, generator=gen, **dev),
        "frequency": 0.5 * torch.rand(requests, generator=gen, **dev),
        "request": None, "row_lens": None, "bias_offsets": None, "bias_ids": None, "bias_values": None,
        "mask": None, "mask_index": None,
    }
    if per > 1:  # the rows of a request's drafts: row q sees q tokens more of the history
        row = torch.arange(rows, **dev)
        state["request"] = (row // per).to(torch.int32)
        state["row_lens"] = (seq[row // per] - per + 1 + row % per).clamp(min=0).to(torch.int32)
    if case["bias"]:
        b = case["bias"]
        state["bias_offsets"] = (torch.arange(requests + 1, **dev) * b).to(torch.int32)
        first = torch.randint(vocab, (requests, 1), generator=gen, **dev)
        step = torch.randint(1, vocab // b, (requests, b), generator=gen, **dev).cumsum(1)
        state["bias_ids"] = ((first + step) % vocab).to(torch.int32).reshape(-1)
        state["bias_values"] = torch.empty(requests * b, **dev).normal_(0.0, 4.0, generator=gen)
    if case["mask"]:  # three quarters of the rows under a grammar: some states allow little, some nearly all
        words = -(-vocab // 32)
        few = torch.zeros(rows, words * 32, dtype=torch.bool, **dev)
        few.scatter_(1, torch.randint(vocab, (rows, 200), generator=gen, **dev), True)
        allowed = few ^ (torch.rand(rows, 1, generator=gen, **dev) < 0.5)
        allowed = allowed.view(rows, words, 32)
        packed = torch.zeros(rows, words, dtype=torch.int64, **dev)
        for bit in range(32):
            packed |= allowed[:, :, bit].long() << bit
        state["mask"] = torch.where(packed >= 1 << 31, packed - (1 << 32), packed).to(torch.int32)
        row = torch.arange(rows, **dev)
        state["mask_index"] = torch.where(row % 4 == 3, -1, row).to(torch.int32)
    return state


def _distill_state(case, gen):
    rows, vocab, k = case["rows"], case["vocab"], case["k"]
    logits = _logits(case, rows, gen)
    # a student that has some way to go: the teacher's logits are its own, flatter and under noise
    teacher = torch.empty(rows, vocab, device="cuda").normal_(0.0, 2.0, generator=gen)
    teacher += 0.7 * logits.float()
    teacher /= case["temperature"]
    top, ids = teacher.topk(k, dim=1)
    top = top - teacher.logsumexp(1, keepdim=True)
    row = torch.arange(rows, device="cuda")
    weights = torch.where(row % 8 == 7, 0.0, 1.0 / rows)  # positions of the prompt count nothing
    return {"logits": logits, "ids": ids.to(torch.int32), "log_probs": top.float().contiguous(), "weights": weights,
            "grad_loss": torch.rand(rows, device="cuda", generator=gen) + 0.5}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if case["op"] == "process":
        state = _process_state(case, gen)
    elif case["op"] == "top":
        logits, gather = _source(case, case["rows"], gen)
        state = {"logits": logits, "gather": gather}
    else:
        state = _distill_state(case, gen)
    state["case"] = case
    if own and case["op"] == "process":  # the requests' parameters, as a serving program keeps them
        import logits_sampling_gb300 as ls
        state["params"] = ls.LogitsParams(
            tokens=state["tokens"], prompt_lens=state["prompt_lens"], seq_lens=state["seq_lens"],
            repetition_penalty=state["repetition"], presence_penalty=state["presence"],
            frequency_penalty=state["frequency"], bias_offsets=state["bias_offsets"], bias_ids=state["bias_ids"],
            bias_values=state["bias_values"])
    return state


# -- the calls of the package ---------------------------------------------------


def _run_own(state):
    import logits_sampling_gb300 as ls
    case = state["case"]
    if case["op"] == "process":
        return ls.process_logits(state["logits"], case["rows"], state["params"], gather_indices=state["gather"],
                                 token_to_request_index=state["request"], row_lens=state["row_lens"],
                                 allowed_mask=state["mask"], mask_index=state["mask_index"])
    if case["op"] == "top":
        return ls.top_log_probs(state["logits"], case["k"], n=case["rows"], temperature=case["temperature"],
                                gather_indices=state["gather"])
    teacher = (state["ids"], state["log_probs"])
    how = {"temperature": case["temperature"], "tail": case["tail"], "weights": state["weights"]}
    if case["way"] == "loss":
        loss, _ = ls.distill_loss(state["logits"], *teacher, **how)
        return loss
    if case["way"] == "step":
        loss, stats = ls.distill_loss(state["logits"], *teacher, **how)
        return loss, ls.distill_loss_backward(state["logits"], *teacher, stats, grad_loss=state["grad_loss"], **how)
    return ls.distill_loss_grad(state["logits"], *teacher, **how)


# -- the plain forms ------------------------------------------------------------


def _rows_of(state, case):
    x = state["logits"] if state["gather"] is None else state["logits"][state["gather"].long()]
    return x.float()


def _plain_process(state):
    case = state["case"]
    rows, vocab = case["rows"], case["vocab"]
    x = _rows_of(state, case)
    request = torch.arange(rows, device="cuda") if state["request"] is None else state["request"].long()
    tokens = state["tokens"][request].long()
    length = (state["seq_lens"][request] if state["row_lens"] is None else state["row_lens"]).long()[:, None]
    prompt = state["prompt_lens"][request].long()[:, None]
    at = torch.arange(tokens.shape[1], device="cuda")[None, :]
    here = (at < length) & (tokens >= 0) & (tokens < vocab)
    count = torch.zeros(rows, vocab + 1, device="cuda")  # the last column takes what does not count
    count.scatter_add_(1, torch.where(here & (at >= prompt), tokens, vocab), torch.ones_like(tokens, dtype=torch.float32))
    seen = torch.zeros(rows, vocab + 1, dtype=torch.bool, device="cuda")
    seen.scatter_(1, torch.where(here, tokens, vocab), True)
    count, seen = count[:, :vocab], seen[:, :vocab]
    rho = state["repetition"][request][:, None]
    y = torch.where(seen, torch.where(x > 0, x / rho, x * rho), x)
    y = y - state["frequency"][request][:, None] * count
    y = y - state["presence"][request][:, None] * (count > 0)
    if state["bias_ids"] is not None:
        b = case["bias"]
        ids = state["bias_ids"].view(-1, b)[request].long()
        y.scatter_add_(1, ids, state["bias_values"].view(-1, b)[request])
    if state["mask"] is not None:
        which = state["mask_index"].long()
        words = state["mask"][which.clamp(min=0)]
        bits = (words[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        allowed = (bits.view(rows, -1)[:, :vocab] != 0) | (which < 0)[:, None]
        y = torch.where(allowed, y, -math.inf)
    return y.to(state["logits"].dtype)


def _plain_top(state):
    case = state["case"]
    x = _rows_of(state, case)
    z = x / case["temperature"]
    m = z.amax(1, keepdim=True)
    lse = m + (z - m).exp().sum(1, keepdim=True).log()
    # distinct 64-bit keys: the value's order first, then the lower index
    b = x.view(torch.int32).long()
    order = torch.where(b >= 0, b, -(b & 0x7FFFFFFF))
    key = (order << 32) - torch.arange(x.shape[1], device="cuda")
    best = key.topk(case["k"], dim=1).indices
    return best.to(torch.int32), z.gather(1, best) - lse, lse[:, 0]


def _plain_distill(state):
    case = state["case"]
    x, tau, tail = state["logits"], case["temperature"], case["tail"]
    rows, vocab = x.shape
    z = x.float() / tau
    ids, t, w = state["ids"].long(), state["log_probs"], state["weights"]
    valid = (ids >= 0) & (ids < vocab)
    at = torch.where(valid, ids, 0)
    p = torch.where(valid, t.exp(), 0.0)
    mass = p.sum(1, keepdim=True)
    in_top = torch.zeros(rows, vocab + 1, dtype=torch.bool, device="cuda")
    in_top = in_top.scatter_(1, torch.where(valid, ids, vocab), True)[:, :vocab]
    m = z.amax(1, keepdim=True)
    e = (z - m).exp()
    s = e.sum(1, keepdim=True)
    if tail == "renorm":
        p, t, mass = p / mass, t - mass.log(), torch.ones_like(mass)
    kl = torch.where(p > 0, p * (t - (z.gather(1, at) - m - s.log())), 0.0).sum(1)
    scale = mass
    if tail == "bucket":
        zr = torch.where(in_top, -math.inf, z)
        mr = zr.amax(1, keepdim=True)
        er = (zr - mr).exp()
        sr = er.sum(1, keepdim=True)
        pr = (1 - mass).clamp(min=0)
        kl = kl + torch.where(pr > 0, pr * (pr.log() - (mr - m + (sr / s).log())), 0.0)[:, 0]
        scale = mass + pr
    loss = torch.where(w != 0, w * kl, 0.0)
    if case["way"] == "loss":
        return loss
    g = w if case["way"] == "fused" else w * state["grad_loss"]
    d = e * (scale / s)
    if tail == "bucket":
        d = d - er * (pr / sr)
    d.scatter_add_(1, at, -p)
    d = torch.where((g != 0)[:, None], d * (g / tau)[:, None], 0.0)
    return loss, d.to(x.dtype)


def run(state):
    if own:
        return _run_own(state)
    return {"process": _plain_process, "top": _plain_top, "distill": _plain_distill}[state["case"]["op"]](state)


# -- the work that a pass cannot do without ---------------------------------------


def work(case):
    rows, vocab, size = case["rows"], case["vocab"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "process":
        cap = case["history"]
        mean = (cap - 16) / max(math.log(cap / 16), 1e-9) if cap > 16 else cap  # of the lengths drawn over their logarithm
        requests = -(-rows // case["per_request"])
        moved = 2 * rows * vocab * size + requests * (4 * mean + 8 * case["bias"] + 20)
        if case["mask"]:
            moved += (rows - rows // 4) * vocab / 8
        return {"bytes": moved, "flops": rows * (mean + case["bias"]) * 4}
    k = case["k"]
    if case["op"] == "top":
        return {"bytes": rows * (vocab * size + 8 * k + 4), "flops": 3 * rows * vocab}
    read = (rows - rows // 8) * (vocab * size + 8 * k) + 8 * rows  # a row of no weight is not read
    if case["way"] == "loss":
        return {"bytes": read, "flops": 3 * rows * vocab}
    return {"bytes": read + rows * vocab * size, "flops": 6 * rows * vocab}


# -- the definitions in 64 bits -----------------------------------------------------


def _exact_process(s, case):
    rows, vocab = case["rows"], case["vocab"]
    src = s["gather"].tolist() if s["gather"] is not None else range(rows)
    request = s["request"].tolist() if s["request"] is not None else range(rows)
    out = []
    lens = (s["row_lens"] if s["row_lens"] is not None else s["seq_lens"]).tolist()
    prompt = s["prompt_lens"].tolist()
    rep, pres, freq = (s[n].double() for n in ("repetition", "presence", "frequency"))
    place = torch.arange(vocab, device="cuda")
    for i, (row, r) in enumerate(zip(src, request)):
        x = s["logits"][row].double()
        text = s["tokens"][r, :lens[i]].long()
        said = torch.bincount(text[min(prompt[r], lens[i]):], minlength=vocab).double()
        any_ = torch.bincount(text, minlength=vocab) > 0
        y = x.clone()
        y[any_ & (x > 0)] /= rep[r]
        y[any_ & (x <= 0)] *= rep[r]
        y -= freq[r] * said + pres[r] * said.clamp(max=1.0)
        if case["bias"]:
            lo, hi = r * case["bias"], (r + 1) * case["bias"]
            y[s["bias_ids"][lo:hi].long()] += s["bias_values"][lo:hi].double()
        if case["mask"] and int(s["mask_index"][i]) >= 0:
            word = s["mask"][i].long()[place // 32]
            y[(word >> (place % 32)) % 2 == 0] = -math.inf
        out.append(y.to(torch.float32) if rows * vocab > 1 << 26 else y)
    return torch.stack(out)


def _exact_top(s, case):
    lp, total = [], []
    for i in range(case["rows"]):
        z = s["logits"][i if s["gather"] is None else int(s["gather"][i])].double() / case["temperature"]
        a = torch.logsumexp(z, 0)
        total.append(a)
        lp.append(torch.sort(z, descending=True).values[:case["k"]] - a)
    return [None, torch.stack(lp), torch.stack(total)]


def _exact_distill(s, case):
    tau, k = case["temperature"], case["k"]
    losses, grads = [], []
    for i in range(case["rows"]):
        w = float(s["weights"][i])
        up = w if case["way"] == "fused" else w * float(s["grad_loss"][i])
        log_q = torch.log_softmax(s["logits"][i].double() / tau, 0)
        at, log_p = s["ids"][i].long(), s["log_probs"][i].double()
        if case["tail"] == "renorm":
            log_p = torch.log_softmax(log_p, 0)
        p = log_p.exp()
        target = torch.zeros_like(log_q)
        target[at] = p
        loss = (p * (log_p - log_q[at])).sum()
        d = log_q.exp() * p.sum() - target
        if case["tail"] == "bucket":
            others = torch.ones_like(log_q, dtype=torch.bool)
            others[at] = False
            rest_q = torch.logsumexp(log_q[others], 0)
            rest_p = torch.clamp(1 - p.sum(), min=0)
            if float(rest_p) > 0:
                loss = loss + rest_p * (rest_p.log() - rest_q)
                d = d + rest_p * log_q.exp()
                d[others] -= rest_p * (log_q[others] - rest_q).exp()
        losses.append(w * loss)
        if case["way"] != "loss":
            d = d * (up / tau)
            grads.append(d.to(torch.float32) if case["rows"] * case["vocab"] > 1 << 26 and case["dtype"] == "bf16" else d)
    loss = torch.stack(losses)
    return loss if case["way"] == "loss" else [loss, torch.stack(grads)]


def exact(case, seed):
    state = prepare(case, seed)
    return {"process": _exact_process, "top": _exact_top, "distill": _exact_distill}[case["op"]](state, case)
