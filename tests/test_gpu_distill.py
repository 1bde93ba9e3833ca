"""GPU checks of the distillation loss and its gradient against their
definitions in 64 bits, and of the gradient against differences of the loss."""
import numpy as np
import pytest

import row_ops_ref as R

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "bf16"]
TAILS = ["drop", "renorm", "bucket"]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    import logits_sampling_gb300 as ls
    ls.load_library()


def _dev(v, t):
    import torch
    return None if v is None else torch.from_numpy(np.ascontiguousarray(v, t)).cuda()


def _targets(rng, x, k, T, noise=1.5):
    """A teacher's top k under noise around the student, as float32."""
    n, V = x.shape
    z = (np.nan_to_num(x, nan=-30.0, posinf=30.0, neginf=-30.0) + rng.standard_normal((n, V)) * noise) / T
    m = z.max(1, keepdims=True)
    lse = m + np.log(np.exp(z - m).sum(1, keepdims=True))
    ids = np.argsort(-z, 1, kind="stable")[:, :k].astype(np.int32)
    return ids, (np.take_along_axis(z, ids, 1) - lse).astype(np.float32)


def _calls(x, dev, ids, lp, T, tail, w, g):
    """Loss and gradient by every entry point; the ways must agree."""
    import torch
    import logits_sampling_gb300 as ls
    ids_d, lp_d, w_d, g_d = _dev(ids, np.int32), _dev(lp, np.float32), _dev(w, np.float32), _dev(g, np.float32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    how = {"temperature": T, "tail": tail, "weights": w_d}
    loss, stats = ls.distill_loss(dev, ids_d, lp_d, error_word=err, **how)
    grad = ls.distill_loss_backward(dev, ids_d, lp_d, stats, grad_loss=g_d, **how)
    loss2, grad2 = ls.distill_loss_grad(dev, ids_d, lp_d, error_word=err, **how)
    f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    return f(loss), f(grad), f(loss2), f(grad2), int(err.item())


def _check(x, ids, lp, T, tail, w, g, got, dtype, where=""):
    loss, grad, loss2, grad2, _ = got
    n = len(x)
    for i in range(n):
        wi = 1.0 if w is None else float(np.float32(w[i]))
        gi = 1.0 if g is None else float(np.float32(g[i]))
        for L, D, up in ((loss, grad, gi), (loss2, grad2, 1.0)):
            rl, tl, rd, td = R.distill_row(x[i], ids[i], lp[i], T, tail, wi, up)
            if np.isnan(rl):
                assert np.isnan(L[i]) and np.isnan(D[i]).all(), (where, i)
                continue
            if np.isinf(rl):
                assert L[i] == rl, (where, i, L[i], rl)
            else:
                assert abs(L[i] - rl) <= tl, (where, i, tail, L[i], rl, tl)
            ok = R.within(D[i], rd, td, dtype)
            assert ok.all(), (where, i, tail, np.nonzero(~ok)[0][:4], D[i][~ok][:4], rd[~ok][:4], td[~ok][:4])


@pytest.mark.parametrize("tail", TAILS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V,k", [(2, 1), (5, 5), (31, 7), (300, 256), (1001, 8), (4097, 1), (32003, 64),
                                 (128256, 64), (151936, 20), (262144, 128)])
def test_against_the_definition(tail, dtype, V, k):
    rng = np.random.default_rng(V + k)
    n = 4
    x = R.to_dtype(rng.standard_normal((n, V)) * 3, dtype)
    w = np.array([0.5, 0.0, 1.0, -2.0], np.float32)
    g = np.array([1.0, 3.0, 0.7, 0.1], np.float32)
    for T in (1.0, 2.0):
        ids, lp = _targets(rng, x, k, T)
        got = _calls(x, R.device_matrix(x, dtype), ids, lp, T, tail, w, g)
        _check(x, ids, lp, T, tail, w, g, got, dtype, f"T={T}")
        assert got[4] == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 9, 80, 400])
def test_batch_sizes(dtype, rows):
    rng = np.random.default_rng(rows)
    x = R.to_dtype(rng.standard_normal((rows, 5003)) * 3, dtype)
    ids, lp = _targets(rng, x, 20, 1.0)
    _check(x, ids, lp, 1.0, "bucket", None, None, _calls(x, R.device_matrix(x, dtype), ids, lp, 1.0, "bucket", None, None),
           dtype)


@pytest.mark.parametrize("tail", TAILS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("col_off,pad,out_off", [(1, 0, 0), (3, 5, 3), (7, 1, 2), (8, 8, 0)])
def test_strides_and_alignments(tail, dtype, col_off, pad, out_off):
    import torch
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(col_off)
    n, V, k = 5, 9001, 30
    x = R.to_dtype(rng.standard_normal((n, V)) * 3, dtype)
    ids, lp = _targets(rng, x, k, 1.0)
    dev = R.device_matrix(x, dtype, col_off, pad)
    wide = torch.zeros((n, k + 3), dtype=torch.float32, device="cuda")
    wide[:, :k] = _dev(lp, np.float32)
    wide_ids = torch.zeros((n, k + 3), dtype=torch.int32, device="cuda")
    wide_ids[:, :k] = _dev(ids, np.int32)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    whole = torch.full((n, out_off + V + 5), 7.0, dtype=t, device="cuda")
    out = whole[:, out_off:out_off + V]
    loss, stats = ls.distill_loss(dev, wide_ids[:, :k], wide[:, :k], tail=tail)
    f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    ls.distill_loss_backward(dev, wide_ids[:, :k], wide[:, :k], stats, tail=tail, out=out)
    a = f(out)
    whole.fill_(7.0)
    loss2, _ = ls.distill_loss_grad(dev, wide_ids[:, :k], wide[:, :k], tail=tail, out_grad=out)
    _check(x, ids, lp, 1.0, tail, None, None, (f(loss), a, f(loss2), f(out), 0), dtype)
    side = torch.cat([whole[:, :out_off], whole[:, out_off + V:]], 1)
    assert bool((side == 7.0).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1001, 50001])
def test_gradient_over_the_logits(dtype, V):
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(5)
    x = R.to_dtype(rng.standard_normal((6, V)) * 3, dtype)
    ids, lp = _targets(rng, x, 12, 1.0)
    ids_d, lp_d = _dev(ids, np.int32), _dev(lp, np.float32)
    a, b = R.device_matrix(x, dtype, 3, 2), R.device_matrix(x, dtype, 3, 2)
    loss, stats = ls.distill_loss(a, ids_d, lp_d)
    ref = ls.distill_loss_backward(a, ids_d, lp_d, stats).float().cpu().numpy()
    ls.distill_loss_backward(a, ids_d, lp_d, stats, out=a)
    loss2, _ = ls.distill_loss_grad(b, ids_d, lp_d, out_grad=b)
    assert np.array_equal(a.float().cpu().numpy(), ref)
    _check(x, ids, lp, 1.0, "bucket", None, None,
           (loss.cpu().numpy(), ref.astype(np.float64), loss2.cpu().numpy(), b.float().cpu().numpy().astype(np.float64),
            0), dtype)


@pytest.mark.parametrize("tail", TAILS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_special_values(tail, dtype):
    """Masked logits, NaN, infinities, the type's lowest value; padded and empty targets."""
    import torch
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(11)
    n, V, k = 12, 700, 9
    x = (rng.standard_normal((n, V)) * 2).astype(np.float32)
    x = R.to_dtype(x, dtype)
    ids, lp = _targets(rng, x, k, 1.0)
    x[0, ids[0, 3]] = -np.inf          # the student forbids one of the teacher's ids: infinite loss
    x[1, 300:] = -np.inf               # masked student, targets within
    ids[1] = np.arange(k) * 7
    x[2, ::7] = np.nan
    x[3, :] = -np.inf                  # nothing left
    x[4, :] = -np.inf                  # mass on the targets alone: no tail
    x[4, ids[4]] = np.linspace(-1, 1, k)
    x[5, :] = float(torch.finfo(torch.bfloat16).min)
    x[5, ids[5]] = 0.0                 # the tail's mass underflows against the head's
    ids[6, 4:] = -1                    # padding
    lp[7, 5:] = -np.inf
    ids[8, :] = V + 5                  # no target at all
    lp[9, 2] = np.nan
    x[10, 500] = np.inf                # outside the targets' reach or in it
    x[11, ids[11, 0]] = np.inf
    ids[10][ids[10] == 500] = 501 if 501 not in ids[10] else 502
    x = R.to_dtype(x, dtype)
    got = _calls(x, R.device_matrix(x, dtype), ids, lp, 1.0, tail, None, None)
    rows = [i for i in range(n)]
    _check(x[rows], ids[rows], lp[rows], 1.0, tail, None, None, got, dtype)
    assert got[4] == ls.LS_ROW_ERR_NO_FINITE


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [3001, 120001])
def test_stretches_of_nan(dtype, V):
    """NaN logits are -inf wherever they lie: alone, in whole stretches, beside
    -inf, at the targets, up to a row of nothing else."""
    rng = np.random.default_rng(V)
    x = (rng.standard_normal((7, V)) * 2).astype(np.float32)
    x = R.to_dtype(x, dtype)
    ids, lp = _targets(rng, x, 9, 1.0)
    x[0, : V // 2] = np.nan
    x[1, V // 3:] = np.nan
    x[2, :] = np.nan
    x[2, V - 5] = 1.0
    x[3, : V // 2] = -np.inf
    x[3, : V // 2: 3] = np.nan
    x[4, ids[4]] = np.nan
    x[5, :] = np.nan
    x[6, 7] = np.nan
    for tail in TAILS:
        got = _calls(x, R.device_matrix(x, dtype, 1, 2), ids, lp, 1.0, tail, None, None)
        _check(x, ids, lp, 1.0, tail, None, None, got, dtype)


def test_weight_zero_is_not_read():
    import torch
    import logits_sampling_gb300 as ls
    x = torch.full((3, 1000), float("nan"), device="cuda")
    ids = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    ids[:, 1] = 4
    lp = torch.full((3, 2), -1.0, device="cuda")
    w = torch.zeros(3, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, stats = ls.distill_loss(x, ids, lp, weights=w, error_word=err)
    grad = ls.distill_loss_backward(x, ids, lp, stats, weights=w)
    loss2, grad2 = ls.distill_loss_grad(x, ids, lp, weights=w, error_word=err)
    for t in (loss, grad, loss2, grad2, err):
        assert bool((t == 0).all())
    assert ls.distill_loss(x[:0], ids[:0], lp[:0])[0].shape == (0,)


@pytest.mark.parametrize("tail", TAILS)
def test_gradient_against_differences_of_the_loss(tail):
    """Central differences of the fp32 loss along random directions.  With step h
    the difference holds h^2 / 6 times the third derivative (at most 1 for a
    direction of unit largest entry over T = 1) and the loss's rounding over h:
    at h = 1/64, 4e-5 + 64 * 4e-6."""
    rng = np.random.default_rng(21)
    V, k, h = 50, 6, 1.0 / 64
    x = R.to_dtype(rng.standard_normal((1, V)) * 2, "f32")
    ids, lp = _targets(rng, x, k, 1.0)
    _, grad, _, grad2, _ = _calls(x, R.device_matrix(x, "f32"), ids, lp, 1.0, tail, None, None)
    for _ in range(8):
        d = rng.choice([-1.0, 0.0, 1.0], V)
        up = _calls(x, R.device_matrix((x + h * d).astype(np.float32), "f32"), ids, lp, 1.0, tail, None, None)[0][0]
        dn = _calls(x, R.device_matrix((x - h * d).astype(np.float32), "f32"), ids, lp, 1.0, tail, None, None)[0][0]
        diff = (up - dn) / (2 * h)
        for gr in (grad, grad2):
            assert abs(diff - float((gr[0] * d).sum())) <= 5e-4, (diff, float((gr[0] * d).sum()))


@pytest.mark.parametrize("dtype", DTYPES)
def test_autograd(dtype):
    """ls.distill as a node of a graph: the gradient reaches what made the logits."""
    import torch
    import logits_sampling_gb300 as ls
    rng = np.random.default_rng(2)
    x = R.to_dtype(rng.standard_normal((4, 3000)), dtype)
    ids, lp = _targets(rng, x, 10, 2.0)
    dev = R.device_matrix(x, dtype).contiguous().requires_grad_()
    loss = ls.distill(dev * 1.0, _dev(ids, np.int32), _dev(lp, np.float32), temperature=2.0, tail="renorm")
    up = torch.tensor([1.0, 2.0, 0.5, 0.0], device="cuda")
    (loss * up).sum().backward()
    g = dev.grad.float().cpu().numpy().astype(np.float64)
    for i in range(4):
        _, _, rd, td = R.distill_row(x[i], ids[i], lp[i], 2.0, "renorm", 1.0, float(up[i]))
        assert R.within(g[i], rd, td, dtype).all()


def test_offsets_past_32_bits():
    import torch
    import logits_sampling_gb300 as ls
    V, rows = 262144, 16640
    x = torch.zeros((rows, V), dtype=torch.bfloat16, device="cuda")
    x[-2:] = (torch.randn(2, V, device="cuda") * 3).to(torch.bfloat16)
    host = x[-2:].float().cpu().numpy()
    ids, lp = _targets(np.random.default_rng(1), host, 16, 1.0)
    all_ids = torch.arange(16, dtype=torch.int32, device="cuda").repeat(rows, 1)
    all_lp = torch.full((rows, 16), -3.0, device="cuda")
    all_ids[-2:] = _dev(ids, np.int32)
    all_lp[-2:] = _dev(lp, np.float32)
    f = lambda t: t[-2:].float().cpu().numpy().astype(np.float64)  # noqa: E731
    loss, stats = ls.distill_loss(x, all_ids, all_lp)
    grad = f(ls.distill_loss_backward(x, all_ids, all_lp, stats))
    loss2, grad2 = ls.distill_loss_grad(x, all_ids, all_lp, out_grad=x)
    _check(host, ids, lp, 1.0, "bucket", None, None, (f(loss), grad, f(loss2), f(grad2), 0), "bf16")


@pytest.mark.parametrize("dtype", DTYPES)
def test_largest_vocab(dtype):
    import logits_sampling_gb300 as ls
    V = ls.row_ops_max_vocab(ls.LS_DTYPE_BF16)
    rng = np.random.default_rng(0)
    x = R.to_dtype(rng.standard_normal((1, V)) * 3, dtype)
    ids, lp = _targets(rng, x, 40, 1.0)
    got = _calls(x, R.device_matrix(x, dtype, 1, 1), ids, lp, 1.0, "bucket", None, None)
    _check(x, ids, lp, 1.0, "bucket", None, None, got, dtype)
    with pytest.raises(ls.LSError):
        ls.distill_loss(R.device_matrix(np.zeros((1, V + 1)), dtype), _dev(ids, np.int32), _dev(lp, np.float32))


def test_same_bits_every_time_on_any_stream():
    import torch
    import logits_sampling_gb300 as ls
    x = (torch.randn(200, 32000, device="cuda") * 3).to(torch.bfloat16)
    ids, lp, _ = ls.top_log_probs((x.float() + torch.randn_like(x.float())).to(torch.bfloat16), 32)
    a = ls.distill_loss_grad(x, ids, lp)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = ls.distill_loss_grad(x, ids, lp, stream=s)
    s.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    loss, grad = torch.zeros_like(a[0]), torch.zeros_like(a[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ls.distill_loss_grad(x, ids, lp, out_loss=loss, out_grad=grad)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a[0], loss) and torch.equal(a[1], grad)
