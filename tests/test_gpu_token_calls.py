"""Calls of the operators on sampled tokens that their documentation allows and
the tests of their values do not make: outputs given by the caller, in place for
every layout of a batch, empty and far-apart rows, temperatures at which a long
row leaves the fast path, refusals on the device."""
import numpy as np
import pytest

from test_gpu_token_ops import _check_gradient, _dev, _f64, _logits, _near, _normal, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


def _batch(n, V, dtype, seed=0):
    rng = np.random.default_rng(seed)
    dev, x = _logits(_normal(rng, n, V), dtype, 3, 6)
    return dev, x, rng.integers(0, V, n), _dev(rng.standard_normal(n)), rng


def test_outputs_of_the_caller():
    """They are filled and returned, count as changed in place, and autograd refuses what it saved of them."""
    import logits_sampling_gb300 as ls
    import torch
    n, V = 9, 700
    x, _, ids, adv, _ = _batch(n, V, "f32")
    ids = _dev(ids, np.int32)
    off = _dev([0, 3, 9], np.int32)

    def empty(*shape):
        return torch.full(shape, 9.0, device="cuda")

    for call, args, names in (
            (ls.token_log_probs, (x, ids), {"out": (n,), "out_entropy": (n,), "out_stats": (n, ls.TOKEN_STATS)}),
            (ls.policy_loss, (x, ids, adv), {"out": (n,), "out_metrics": (n, 4), "out_stats": (n, ls.TOKEN_STATS)}),
            (ls.policy_loss_grad, (x, ids, adv), {"out_loss": (n,), "out_grad": (n, V), "out_metrics": (n, 4)}),
            (ls.preference_loss, (x, ids, off), {"out": (1,), "out_log_ratios": (2,), "out_stats": (n, ls.TOKEN_STATS)})):
        given = {k: empty(*s) for k, s in names.items()}
        versions = {k: t._version for k, t in given.items()}
        got = call(*args, **given)
        new = call(*args, entropy=True) if call is ls.token_log_probs else call(*args)
        assert all(a is b for a, b in zip(got, given.values())), call
        assert all(given[k]._version > versions[k] for k in given), call
        # stats hold NaN where no entropy was asked for
        assert all(torch.allclose(a, b, rtol=0, atol=0, equal_nan=True) for a, b in zip(got, new)), call
        with torch.inference_mode():
            inside = call(*args)
            assert all(a is None or a.is_inference() for a in inside)
    _, _, stats = ls.token_log_probs(x, ids)
    out = empty(n, V)
    assert ls.token_log_probs_backward(x, ids, stats, adv, out=out) is out
    leaf = x.clone().requires_grad_()
    held = leaf * 1.0
    lp, _ = ls.score(held, ids)
    ls.policy_loss_grad(held.detach(), ids, adv, out_grad=held.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        lp.sum().backward()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", [(3, 128256), (100, 9001), (200, 40001), (700, 3001), (650, 20001), (130, 100001),
                                 (129, 200003)])
def test_in_place_for_every_layout(dtype, n, V):
    import logits_sampling_gb300 as ls
    import torch
    x, _, ids, adv, _ = _batch(n, V, dtype)
    ids = _dev(ids, np.int32)
    ids[n // 2] = -1
    w = torch.ones(n, device="cuda")
    w[n // 3] = 0
    for how in ({}, {"entropy_coef": 0.1}):
        loss, metrics, stats = ls.policy_loss(x, ids, adv, weights=w, **how)
        want = ls.policy_loss_backward(x, ids, stats)
        loss1, grad1, metrics1 = ls.policy_loss_grad(x, ids, adv, weights=w, **how)
        assert torch.allclose(loss, loss1, rtol=1e-5, atol=1e-5) and torch.allclose(metrics, metrics1, rtol=1e-5, atol=1e-5)
        step = 2.0 ** -6 if dtype == "bf16" else 2e-5
        assert torch.allclose(grad1.float(), want.float(), rtol=step, atol=1e-7)
        for f in (lambda y: ls.policy_loss_grad(y, ids, adv, weights=w, out_grad=y, **how)[1],
                  lambda y: ls.policy_loss_backward(y, ids, stats, out=y)):
            y, _ = _logits(np.zeros((n, V), np.float32), dtype, 3, 6)
            y.copy_(x)
            out = f(y)
            assert out is y and (torch.equal(y, grad1) or torch.equal(y, want))
            around = y.as_strided((n, 6), (V + 6, 1), y.storage_offset() + V)
            assert (around == 77).all()  # the padding between the rows is as it was


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", [(50, 2003), (400, 30001), (7, 70003)])
def test_in_place_where_rows_touch(dtype, n, V):
    """Contiguous rows of odd length share their first and last 32 bytes with their neighbours."""
    import logits_sampling_gb300 as ls
    import torch
    rng = np.random.default_rng(4)
    x, _ = _logits(_normal(rng, n, V), dtype)
    ids, adv = _dev(rng.integers(0, V, n), np.int32), _dev(rng.standard_normal(n))
    ids[::3] = torch.tensor([0, V - 1], device="cuda").repeat(n)[:len(ids[::3])].to(torch.int32)  # at the edges
    want = ls.policy_loss_grad(x, ids, adv)[1]
    _, _, stats = ls.policy_loss(x, ids, adv)
    back = ls.policy_loss_backward(x, ids, stats)
    for f, g in ((lambda y: ls.policy_loss_grad(y, ids, adv, out_grad=y)[1], want),
                 (lambda y: ls.policy_loss_backward(y, ids, stats, out=y), back)):
        for _ in range(3):
            y = x.clone()
            assert torch.equal(f(y), g)


def test_rows_far_apart():
    """Rows that begin past 2^31 entries of their buffer, read and written."""
    import logits_sampling_gb300 as ls
    import torch
    n, V, stride = 3, 5000, 1_200_000_008
    buf = torch.empty(2 * stride + V, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((n, V), (stride, 1))
    near = torch.randn(n, V, device="cuda").to(torch.bfloat16)
    x.copy_(near)
    ids = _dev([0, 17, V - 1], np.int32)
    adv = torch.randn(n, device="cuda")
    off = _dev([0, 1, 3], np.int32)
    a = ls.token_log_probs(x, ids, entropy=True)
    b = ls.token_log_probs(near, ids, entropy=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(*(ls.token_log_probs_backward(y, ids, st, adv, adv) for y, st in ((x, a[2]), (near, b[2]))))
    assert torch.equal(ls.preference_loss(x, ids, off)[0], ls.preference_loss(near, ids, off)[0])
    want = ls.policy_loss_grad(near, ids, adv)
    got = ls.policy_loss_grad(x, ids, adv, out_grad=x)
    assert torch.equal(got[0], want[0]) and torch.equal(x, want[1])


def test_no_rows():
    import logits_sampling_gb300 as ls
    import torch
    x = torch.zeros(0, 100, device="cuda")
    ids, none = _dev(np.zeros(0), np.int32), torch.zeros(0, device="cuda")
    lp, h, stats = ls.token_log_probs(x, ids, entropy=True)
    assert lp.shape == h.shape == (0,) and ls.token_log_probs_backward(x, ids, stats, none, none).shape == (0, 100)
    loss, metrics, stats = ls.policy_loss(x, ids, none)
    assert loss.shape == (0,) and metrics.shape == (0, 4) and ls.policy_loss_backward(x, ids, stats).shape == (0, 100)
    assert ls.policy_loss_grad(x, ids, none)[1].shape == (0, 100)


@pytest.mark.parametrize("T", [1e-30, 1e-5, 0.02, 1e6, 1e25])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_rows_at_far_temperatures(dtype, T):
    import logits_sampling_gb300 as ls
    import torch
    n, V = 140, 40001
    x, xs, ids, adv, rng = _batch(n, V, dtype, 5)
    ids = xs.argmax(1) if T < 1e-3 else ids
    idd = _dev(ids, np.int32)
    at = list(range(0, n, 20))
    T = float(np.float32(T))
    rows = _rows(xs[at], ids[at], T, dtype)
    g, gh = rng.standard_normal(n).astype(np.float32), rng.standard_normal(n).astype(np.float32)
    for entropy in (False, True):
        lp, h, stats = ls.token_log_probs(x, idd, temperature=T, entropy=entropy)
        for k, i in enumerate(at):
            _near(float(lp[i]), rows[k].lp, rows[k].tol_lp, f"lp {i}")
            if entropy:
                _near(float(h[i]), rows[k].H, rows[k].tol_H, f"H {i}")
        grad = ls.token_log_probs_backward(x, idd, stats, _dev(g), _dev(gh) if entropy else None, temperature=T)
        _check_gradient(_f64(grad[at]), rows, g[at], gh[at] if entropy else np.zeros(len(at)), dtype, "gradient")
    loss, grad, _ = ls.policy_loss_grad(x, idd, adv, temperature=T)
    adv = _f64(adv)
    _check_gradient(_f64(grad[at]), rows, -adv[at], np.zeros(len(at)), dtype, "policy gradient",
                    [abs(adv[i]) * 1e-6 for i in at])
    assert torch.isfinite(loss).all()


def test_refusals_on_the_device():
    import logits_sampling_gb300 as ls
    import torch
    x, _, ids, adv, _ = _batch(6, 300, "f32")
    ids = _dev(ids, np.int32)
    _, _, stats = ls.token_log_probs(x, ids)
    with pytest.raises(ls.LSError):
        ls.token_log_probs(x[:1].expand(6, -1), ids)                       # one row in six places
    with pytest.raises(ls.LSError):
        ls.policy_loss(x, ids, adv, kl_coef=0.1)                           # a KL term without a reference
    with pytest.raises(ls.LSError):
        ls.policy_loss(x, ids, adv, out_metrics=torch.empty(25, device="cuda")[1:].view(6, 4))  # 4 bytes off
    with pytest.raises(ls.LSError):                                          # an overlap that is not in place
        ls.token_log_probs_backward(x, ids, stats, adv, out=x.as_strided((6, 300), x.stride(), x.storage_offset() + 1))
    with pytest.raises(ls.LSError):
        ls.preference_loss(x, ids, _dev([0, 2, 4], np.int32), loss="ipo", label_smoothing=0.1)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ls.LSError):
            ls.token_log_probs(x, ids, temperature=bad)
    with pytest.raises(ValueError):
        ls.token_log_probs_backward(x, ids, stats[:, :8].contiguous(), adv)  # stats of another size
    leaf = x.clone().requires_grad_()
    g, = torch.autograd.grad(ls.score(leaf, ids)[0].sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()                                                   # no second derivatives


@pytest.mark.parametrize("op", ["score", "policy", "preference"])
def test_autograd_in_a_captured_graph(op):
    """Forward and backward captured (no eager graph of the leaf is alive then), replayed on new values."""
    import logits_sampling_gb300 as ls
    import torch
    n, V = 12, 2003
    gen = torch.Generator(device="cuda").manual_seed(9)
    leaf = torch.empty(n, V, device="cuda").normal_(generator=gen).requires_grad_()
    ids = torch.randint(V, (n,), generator=gen, device="cuda").to(torch.int32)
    adv = torch.empty(n, device="cuda").normal_(generator=gen)
    off = _dev([0, 4, 7, 9, 12], np.int32)

    def total():
        if op == "score":
            lp, h = ls.score(leaf, ids, entropy=True)
            return (adv * lp).sum() + h.sum()
        return ls.policy(leaf, ids, adv, adv - 6.0)[0].sum() if op == "policy" else ls.preference(leaf, ids, off)[0].sum()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        total().backward()
    torch.cuda.current_stream().wait_stream(side)
    leaf.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        value = total()
        value.backward()
    captured = leaf.grad
    with torch.no_grad():
        leaf.copy_(leaf.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    got, got_grad = value.detach().clone(), captured.clone()
    leaf.grad = None
    want = total()
    want.backward()
    assert torch.equal(got, want.detach()) and torch.equal(got_grad, leaf.grad)
