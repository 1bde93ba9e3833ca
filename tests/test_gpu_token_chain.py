"""The operators on sampled tokens run together with those around the sampler, as
a training step uses them, and the example that does so."""
import importlib.util
import os

import numpy as np
import pytest

import token_ops_ref as R

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_mask_sample_score_and_train(dtype):
    """Rows under masks, one of which allows nothing: its id is -1, and nothing of it counts."""
    import logits_sampling_gb300 as ls
    import torch
    n, V = 48, 5003
    gen = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.empty(n, V, device="cuda").normal_(0.0, 3.0, generator=gen)
    logits = logits.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    words = torch.randint(-2 ** 31, 2 ** 31 - 1, (n, (V + 31) // 32), generator=gen, device="cuda").to(torch.int32)
    words[7] = 0
    x = ls.process_logits(logits, n, allowed_mask=words)
    prm = ls.SamplingParams.from_host([1.0] * n, [0] * n, [1.0] * n, range(n))
    ids, _, picked = ls.sample_log_probs(x, n, prm, 0, True, True, want_log_probs=False)
    assert int(ids[7]) == -1 and int((ids >= 0).sum()) == n - 1
    old, entropy, stats = ls.token_log_probs(x, ids, entropy=True)
    values = x.float().cpu().numpy().astype(np.float64)
    rows = [None if i == 7 else R.Row(values[i], int(ids[i]), 1.0) for i in range(n)]
    for i, row in enumerate(rows):
        if row is None:
            assert float(old[i]) == 0.0 and float(entropy[i]) == 0.0
            continue
        assert abs(float(old[i]) - row.lp) <= row.tol_lp and abs(float(entropy[i]) - row.H) <= row.tol_H
        assert abs(float(old[i] - picked[i])) <= row.tol_lp + 1e-5  # the sampler's own bound on this log-prob
    adv = torch.empty(n, device="cuda").normal_(generator=gen)
    w = torch.full((n,), 1.0 / n, device="cuda")
    loss, metrics, pstats = ls.policy_loss(x, ids, adv, old, weights=w, entropy=True)
    assert (metrics[[i for i in range(n) if i != 7], 3] == 1).all()  # the same sums in the same order
    grad = ls.policy_loss_backward(x, ids, pstats)
    loss2, grad2, _ = ls.policy_loss_grad(x, ids, adv, old, weights=w)
    forbidden = torch.isinf(x)
    for g in (grad, grad2):
        assert not g[forbidden].any() and not g[7].any()
        for i, row in enumerate(rows):
            if row is not None:
                d, tol = row.gradient(-float(adv[i] * w[i]))
                tol = tol + np.abs(d) * (R.HALF_STEP[dtype] + 4 * row.tol_lp)  # the ratio's own error, too
                assert (np.abs(g[i].float().cpu().numpy() - d) <= tol + R.TINY).all(), i
    assert torch.allclose(loss, loss2, atol=1e-6)
    # on the policy that sampled, the gradient of the policy loss is that of -A lp
    by_score = ls.token_log_probs_backward(x, ids, stats, -adv * w)
    assert torch.allclose(by_score.float(), grad.float(), rtol=2 ** -6 if dtype == "bf16" else 1e-5, atol=1e-7)
    offsets = torch.tensor([0, 8, 20, 33, 48], dtype=torch.int32, device="cuda")
    pairs, ratios, qstats = ls.preference_loss(x, ids, offsets, ref_log_probs=old)
    assert float(ratios.abs().max()) < 1e-4 and torch.allclose(pairs, torch.full_like(pairs, float(np.log(2.0))), atol=1e-5)
    g = ls.preference_loss_backward(x, ids, qstats)
    assert not g[7].any() and g[[0, 8, 20, 33]].any(1).all()
    # the same step from a graph
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ls.policy_loss_grad(x, ids, adv, old, weights=w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], loss2) and torch.equal(out[1], grad2)


def _example():
    import sys
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    spec = importlib.util.spec_from_file_location("train_on_samples", os.path.join(ROOT, "examples", "train_on_samples.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs_and_its_gradients():
    """The gradients of the model's weights against the same losses in plain operations in 64 bits.  An entry of a
    gradient of the logits is off by a few 1e-6 of its row's largest, fp32 products over 96 rows by less: 1e-4 of the
    norm is far above both, and far below what a wrong term gives."""
    import torch
    m = _example()
    model, batch = m.main(["--prompts", "4", "--length", "6", "--updates", "2", "--vocab", "3001"])

    def plain(rows, which):
        z = model64(batch["fed"][rows])
        log_q = torch.log_softmax(z, 1)
        lp = log_q.gather(1, batch["ids"][rows].long()[:, None])[:, 0]
        ref = batch["ref"][rows].double()
        if which == "policy":
            r = (lp - batch["old"][rows].double()).exp()
            a = batch["advantages"][rows].double()
            s = torch.minimum(r * a, r.clamp(0.8, 1.28) * a)
            d = ref - lp
            h = -(log_q.exp() * log_q).sum(1)
            return (batch["weights"][rows].double() * (-s + 0.02 * (d.exp() - d - 1) - 0.01 * h)).sum()
        s = (lp - ref).view(-1, 2, 6).sum(2)
        h = 0.1 * (s[:, 0] - s[:, 1])
        sp = torch.nn.functional.softplus
        return (0.95 * sp(-h) + 0.05 * sp(h)).mean()

    import copy
    model64 = copy.deepcopy(model).double()
    everything = torch.arange(len(batch["ids"]), device="cuda")
    for which, mine, rows in (("policy", lambda: m.policy_loss(model, batch)[0], everything),
                              ("preference", lambda: m.preference_loss(model, batch), batch["pair_rows"])):
        model.zero_grad()
        model64.zero_grad()
        got = mine()
        got.backward()
        want = plain(rows, which)
        want.backward()
        value, wanted = float(got.detach()), float(want.detach())
        assert abs(value - wanted) < 1e-5 * max(1.0, abs(wanted))
        for p, q in zip(model.parameters(), model64.parameters()):
            assert float((p.grad.double() - q.grad).norm()) <= 1e-4 * float(q.grad.norm()), which
