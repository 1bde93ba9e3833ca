"""The operators on sampled tokens on a host without a GPU: every call refuses
bad arguments before any CUDA call, tensors and streams of another device
included, and the 64-bit definitions that the GPU tests compare with hold
against differences and closed forms."""
import ctypes

import numpy as np
import pytest
import torch

import logits_sampling_gb300 as ls
import token_ops_ref as R
from test_row_ops_devices import Claimed, Stream

P = ctypes.c_void_p
FAKE, FAR = P(0x10000), P(0x10000000)  # never dereferenced
N, V, I32 = 4, 400, torch.int32
ROWS = {"logits": FAKE, "dt": 1, "V": V, "stride": V, "n": N, "ids": FAKE, "T": 1.0}
BAD_ROWS = ({"n": -1}, {"logits": None}, {"logits": P(0x10001)}, {"dt": 5}, {"V": 0}, {"stride": V - 1}, {"ids": None},
            {"T": 0.0}, {"T": -1.0}, {"T": float("inf")}, {"T": float("nan")}, {"V": 0x7FFFFFFF, "stride": 0x7FFFFFFF})
BAD_GRAD = ({"out": None}, {"out": P(0x10000001)}, {"out_stride": V - 1}, {"out": FAKE, "out_stride": V + 8},
            {"out": P(0x10010)})


@pytest.fixture(scope="module")
def lib():
    from logits_sampling_gb300 import build as b
    b.build()
    from logits_sampling_gb300 import _row_ops
    return _row_ops._lib()


def _head(kw):
    r = {**ROWS, **{k: v for k, v in kw.items() if k in ROWS}}
    return [r["logits"], r["dt"], r["V"], r["stride"], r["n"], r["ids"]], r["T"]


def _refuses(call, *more):
    assert call(n=0) == 0
    for kw in BAD_ROWS + more:
        assert call(**kw) == 1, kw


def test_score_refusals(lib):
    def call(out=FAR, stats=FAR, **kw):
        head, T = _head(kw)
        return lib.ls_token_log_probs(*head, T, out, None, stats, None, None)

    def back(stats=FAKE, out=FAR, out_stride=V, **kw):
        head, T = _head(kw)
        return lib.ls_token_log_probs_backward(*head, T, stats, None, None, out, out_stride, None)

    _refuses(call, {"out": None}, {"stats": None}, {"stats": P(0x10004)})
    _refuses(back, {"stats": None}, {"stats": P(0x10008)}, *BAD_GRAD)


def test_policy_refusals(lib):
    from logits_sampling_gb300._token_ops import _Policy
    inf, nan = float("inf"), float("nan")

    def policy(**kw):
        p = _Policy(0x10000, 0x10000, 0x10000, None, 0.2, 0.2, 0.0, 0.1, 2, 0.0, 0)
        for k, v in kw.items():
            setattr(p, k, v)
        return ctypes.byref(p)

    def loss(p=policy(), out=FAR, metrics=FAR, stats=FAR, **kw):
        head, T = _head(kw)
        return lib.ls_policy_loss(*head, p, T, out, metrics, stats, None, None)

    def both(p=policy(), loss_=FAKE, metrics=FAR, out=FAR, out_stride=V, **kw):
        head, T = _head(kw)
        return lib.ls_policy_loss_grad(*head, p, T, loss_, metrics, out, out_stride, None, None)

    def back(stats=FAKE, out=FAR, out_stride=V, **kw):
        head, T = _head(kw)
        return lib.ls_policy_loss_backward(*head, T, stats, None, out, out_stride, None)

    bad = [{"p": None}] + [{"p": policy(**kw)} for kw in (
        {"advantages": None}, {"clip_low": -0.1}, {"clip_low": 1.5}, {"clip_low": nan}, {"clip_high": -0.1},
        {"clip_high": nan}, {"dual_clip": 0.5}, {"dual_clip": -1.0}, {"dual_clip": inf}, {"dual_clip": nan},
        {"kl_coef": inf}, {"kl_coef": nan}, {"kl": 3}, {"kl": -1}, {"ref_log_probs": None}, {"entropy_coef": nan},
        {"entropy_coef": inf})] + [{"metrics": P(0x10004)}]
    _refuses(loss, *bad, {"out": None}, {"stats": None}, {"stats": P(0x10004)})
    _refuses(both, *bad, {"loss_": None}, *BAD_GRAD)
    _refuses(back, {"stats": None}, {"stats": P(0x10008)}, *BAD_GRAD)


def test_preference_refusals(lib):
    from logits_sampling_gb300._token_ops import _Preference
    inf, nan = float("inf"), float("nan")

    def preference(**kw):
        p = _Preference(0x10000, 2, None, None, 0, 0.1, 0.0, 0.0, 0)
        for k, v in kw.items():
            setattr(p, k, v)
        return ctypes.byref(p)

    def loss(p=preference(), out=FAR, stats=FAR, **kw):
        head, T = _head(kw)
        return lib.ls_preference_loss(*head, p, T, out, None, stats, None, None)

    def back(stats=FAKE, pairs=2, out=FAR, out_stride=V, **kw):
        head, T = _head(kw)
        return lib.ls_preference_loss_backward(*head, T, stats, pairs, None, out, out_stride, None)

    assert loss(n=0, p=preference(pairs=0)) == 0
    for kw in BAD_ROWS + ({"stats": None}, {"stats": P(0x10004)}, {"out": None}, {"p": None}):
        assert loss(**kw) == 1, kw
    for kw in ({"answer_offsets": None}, {"pairs": -1}, {"pairs": 1 << 30}, {"kind": 3}, {"kind": -1}, {"beta": 0.0},
               {"beta": -1.0}, {"beta": inf}, {"beta": nan}, {"label_smoothing": -0.1}, {"label_smoothing": 0.6},
               {"label_smoothing": nan}, {"label_smoothing": 0.1, "kind": 1}, {"label_smoothing": 0.1, "kind": 2},
               {"margin": nan}, {"margin": inf}, {"margin": 0.5, "kind": 2}):
        assert loss(p=preference(**kw)) == 1, kw
    _refuses(back, {"stats": None}, {"stats": P(0x10008)}, {"pairs": -1}, *BAD_GRAD)


def _arguments():
    """Per call: what it needs, and every further tensor that it may be given, all on device 0."""
    x, ids, vec, word = Claimed((N, V)), Claimed((N,), I32), Claimed((N,)), Claimed((1,), I32)
    stats, off, metrics = Claimed((N, 12)), Claimed((5,), I32), Claimed((N, 4))
    rows = {"logits": x, "ids": ids}
    policy = {"old_log_probs": vec, "ref_log_probs": vec, "weights": vec, "out_metrics": metrics, "error_word": word}
    return {
        "token_log_probs": (rows, {"out": vec, "out_entropy": vec, "out_stats": stats, "error_word": word}),
        "token_log_probs_backward": ({**rows, "stats": stats}, {"grad_log_probs": vec, "grad_entropy": vec, "out": x}),
        "policy_loss": ({**rows, "advantages": vec}, {**policy, "out": vec, "out_stats": stats}),
        "policy_loss_backward": ({**rows, "stats": stats}, {"grad_loss": vec, "out": x}),
        "policy_loss_grad": ({**rows, "advantages": vec}, {**policy, "out_loss": vec, "out_grad": x}),
        "preference_loss": ({**rows, "answer_offsets": off}, {"ref_log_probs": vec, "weights": vec, "out": vec,
                                                              "out_log_ratios": vec, "out_stats": stats,
                                                              "error_word": word}),
        "preference_loss_backward": ({**rows, "stats": stats}, {"grad_loss": vec, "out": x}),
    }


CALLS = list(_arguments())


def test_every_call_is_tried(lib):
    from logits_sampling_gb300._token_ops import CALLS as calls
    assert sorted(calls) == sorted(CALLS)


@pytest.mark.parametrize("call", CALLS)
def test_tensors_and_streams_of_another_device_are_refused(lib, call):
    need, more = _arguments()[call]
    for name in (k for k in (*need, *more) if k != "logits"):
        given = {**need, **more}
        given[name] = Claimed(tuple(given[name].shape), given[name].dtype, 1)
        with pytest.raises(ValueError, match=f"{name} is on cuda:1, the logits are on cuda:0"):
            getattr(ls, call)(**given)
    with pytest.raises(ValueError, match="stream is on cuda:1, the logits are on cuda:0"):
        getattr(ls, call)(**need, stream=Stream())


@pytest.mark.parametrize("call", CALLS)
def test_shapes_types_and_missing_arguments_are_refused(lib, call):
    need, more = _arguments()[call]
    f = getattr(ls, call)
    for name in need:
        with pytest.raises(TypeError):
            f(**{k: v for k, v in need.items() if k != name})
        with pytest.raises(TypeError):
            f(**{**need, name: 3})
    with pytest.raises(TypeError, match="unexpected keyword argument 'nothing'"):
        f(**need, nothing=1)
    with pytest.raises(TypeError):
        f(**{**need, "logits": Claimed((N, V), torch.float16)})
    with pytest.raises(ValueError):
        f(**{**need, "logits": torch.zeros(N, V)})  # not on a GPU
    with pytest.raises(ValueError):
        f(**{**need, "logits": Claimed((N, V, 2))})
    for ids in (Claimed((N - 1,), I32), Claimed((N + 1,), I32)):
        with pytest.raises(ValueError):
            f(**{**need, "ids": ids})
    with pytest.raises(TypeError):
        f(**{**need, "ids": Claimed((N,), torch.int64)})
    for name in more:
        if name in ("error_word",) or (call, name) == ("preference_loss_backward", "grad_loss"):
            continue
        short = Claimed((1,) if more[name].dim() == 1 else (1, 1), more[name].dtype)
        with pytest.raises(ValueError):
            f(**{**need, **more, name: short})
    with pytest.raises(TypeError):
        f(**need, temperature="warm")


def test_words_are_refused(lib):
    need, _ = _arguments()["policy_loss"]
    for call in ("policy_loss", "policy_loss_grad"):
        with pytest.raises(ValueError, match="kl must be one of"):
            getattr(ls, call)(**need, kl="k4")
    need, _ = _arguments()["preference_loss"]
    with pytest.raises(ValueError, match="loss must be one of"):
        ls.preference_loss(**need, loss="softmax")
    with pytest.raises(ValueError, match="2 \\* pairs \\+ 1"):
        ls.preference_loss(**{**need, "answer_offsets": Claimed((4,), I32)})


# -- the definitions --------------------------------------------------------------


def _differences(f, x, grad, tol=1e-7):
    for j in range(len(x)):
        d = np.zeros(len(x))
        d[j] = 1e-5
        assert abs((f(x + d) - f(x - d)) / 2e-5 - grad[j]) < tol, j  # h^2 of third differences and 1e-16 / h


def test_score_definition():
    x = np.random.default_rng(0).standard_normal(40) * 2
    for g_lp, g_H in ((1.0, 0.0), (0.0, 1.0), (0.7, -1.3)):
        def f(v):
            r = R.Row(v, 4, 1.7)
            return g_lp * r.lp + g_H * r.H
        _differences(f, x, R.Row(x, 4, 1.7).gradient(g_lp, g_H)[0])
    r = R.Row(np.log([0.5, 0.25, 0.125, 0.125]), 1, 1.0)
    assert abs(r.lp - np.log(0.25)) < 1e-15 and abs(r.H - 1.75 * np.log(2)) < 1e-15


@pytest.mark.parametrize("kw", [{}, {"dual": 2.0}, {"beta": 0.3, "kl": "k1"}, {"beta": 0.3, "kl": "k2"},
                                {"beta": 0.3, "kl": "k3", "eta": 0.2, "w": 0.4}])
def test_policy_definition(kw):
    x = np.random.default_rng(1).standard_normal(30)
    lp = R.Row(x, 7, 0.9).lp
    for A in (1.5, -0.8):
        for old in (lp, lp + 0.1, lp - 0.15, lp + 1.0, lp - 1.0):
            def f(v):
                return R.policy_row(R.Row(v, 7, 0.9), A, old, lp - 0.4, **kw)[0]
            g = R.policy_row(R.Row(x, 7, 0.9), A, old, lp - 0.4, **kw)
            _differences(f, x, R.Row(x, 7, 0.9).gradient(g[2], g[3])[0])
    # closed forms: a ratio of 2 counts 1.2 for a gain and 2 for a loss
    row = R.Row(np.zeros(4), 0, 1.0)
    assert abs(R.policy_row(row, 1.0, np.log(0.125))[0] + 1.2) < 1e-15
    assert abs(R.policy_row(row, -1.0, np.log(0.125))[0] - 2.0) < 1e-15
    assert abs(R.policy_row(row, -1.0, np.log(0.125), dual=1.5)[0] - 1.5) < 1e-15


@pytest.mark.parametrize("how", [{}, {"smoothing": 0.1}, {"kind": "hinge", "margin": 0.2, "beta": 0.5},
                                 {"kind": "ipo", "beta": 0.5, "average": True}])
def test_preference_definition(how):
    rng = np.random.default_rng(2)
    lp, ref, w = -rng.uniform(0, 5, 6), -rng.uniform(0, 5, 6), rng.uniform(0.5, 1.5, 6)
    _, _, g, _ = R.preference_pair(list(lp), ref, w, 0, 2, 6, **how)

    def f(v):
        return R.preference_pair(list(v), ref, w, 0, 2, 6, **how)[0]
    _differences(f, lp, [g[i] for i in range(6)])
    assert abs(R.preference_pair([0.0] * 4, None, np.ones(4), 0, 2, 4)[0] - np.log(2)) < 1e-15
