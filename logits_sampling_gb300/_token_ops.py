"""Python side of include/ls_token_ops.h: log-probs and entropies of given
tokens, the clipped policy loss with a KL term, the preference loss of pairs of
answers, and their gradients.

The calls themselves (CALLS) are functions of the extension module _row_ops_c
(csrc/py/token_ops_py.h), loaded with those of _row_ops.py; score, policy and
preference are autograd functions over them."""
import ctypes

LS_ROW_ERR_BAD_OFFSETS = 16
TOKEN_STATS = 12  # LS_TOKEN_STATS
POLICY_METRICS = ("log_prob", "entropy", "kl", "ratio")  # columns of a policy loss's metrics
CALLS = ("token_log_probs", "token_log_probs_backward", "policy_loss", "policy_loss_backward", "policy_loss_grad",
         "preference_loss", "preference_loss_backward")

_P, _i32t, _i64t, _f32t, _ci = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_int


class _Policy(ctypes.Structure):
    _fields_ = [("advantages", _P), ("old_log_probs", _P), ("ref_log_probs", _P), ("weights", _P), ("clip_low", _f32t),
                ("clip_high", _f32t), ("dual_clip", _f32t), ("kl_coef", _f32t), ("kl", _ci), ("entropy_coef", _f32t),
                ("entropy", _i32t)]


class _Preference(ctypes.Structure):
    _fields_ = [("answer_offsets", _P), ("pairs", _i32t), ("ref_log_probs", _P), ("weights", _P), ("kind", _ci),
                ("beta", _f32t), ("label_smoothing", _f32t), ("margin", _f32t), ("average", _i32t)]


def configure(lib):
    """Declare the C signatures of include/ls_token_ops.h on a loaded library."""
    P, i32, i64, f32, ci = _P, _i32t, _i64t, _f32t, _ci
    rows = [P, ci, i64, i64, i32, P]  # logits, dtype, vocab, row_stride, n, ids
    lib.ls_token_log_probs.argtypes = rows + [f32, P, P, P, P, P]
    lib.ls_token_log_probs_backward.argtypes = rows + [f32, P, P, P, P, i64, P]
    lib.ls_policy_loss.argtypes = rows + [ctypes.POINTER(_Policy), f32, P, P, P, P, P]
    lib.ls_policy_loss_backward.argtypes = rows + [f32, P, P, P, i64, P]
    lib.ls_policy_loss_grad.argtypes = rows + [ctypes.POINTER(_Policy), f32, P, P, P, i64, P, P]
    lib.ls_preference_loss.argtypes = rows + [ctypes.POINTER(_Preference), f32, P, P, P, P, P]
    lib.ls_preference_loss_backward.argtypes = rows + [f32, P, i32, P, P, i64, P]
    for name in CALLS:
        getattr(lib, "ls_" + name).restype = ci
    return lib


def _contiguous(g):
    """A gradient from above as the calls take it."""
    return None if g is None else g.float().contiguous()


_functions = None


def _autograd():
    """The autograd functions, made when torch and the library are first needed."""
    global _functions
    if _functions is not None:
        return _functions
    import torch

    from ._row_ops import calls
    c = calls()
    once = torch.autograd.function.once_differentiable

    class Score(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, ids, temperature, entropy):
            log_probs, h, stats = c.token_log_probs(logits, ids, temperature, entropy)
            ctx.save_for_backward(logits, ids, stats)
            ctx.temperature = temperature
            ctx.set_materialize_grads(False)
            return log_probs, h

        @staticmethod
        @once
        def backward(ctx, grad_log_probs, grad_entropy):
            logits, ids, stats = ctx.saved_tensors
            return c.token_log_probs_backward(logits, ids, stats, _contiguous(grad_log_probs), _contiguous(grad_entropy),
                                              ctx.temperature), None, None, None

    class Policy(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, ids, advantages, old, ref, weights, temperature, clip_low, clip_high, dual_clip, kl_coef,
                    kl, entropy_coef, entropy):
            loss, metrics, stats = c.policy_loss(logits, ids, advantages, old, ref, weights, temperature, clip_low,
                                                 clip_high, dual_clip, kl_coef, kl, entropy_coef, entropy)
            ctx.save_for_backward(logits, ids, stats)
            ctx.temperature = temperature
            ctx.mark_non_differentiable(metrics)
            return loss, metrics

        @staticmethod
        @once
        def backward(ctx, grad_loss, _):
            logits, ids, stats = ctx.saved_tensors
            return (c.policy_loss_backward(logits, ids, stats, _contiguous(grad_loss), ctx.temperature),) + (None,) * 13

    class Preference(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, ids, offsets, ref, weights, temperature, beta, loss, label_smoothing, margin, average):
            value, ratios, stats = c.preference_loss(logits, ids, offsets, ref, weights, temperature, beta, loss,
                                                     label_smoothing, margin, average)
            ctx.save_for_backward(logits, ids, stats)
            ctx.temperature = temperature
            ctx.mark_non_differentiable(ratios)
            return value, ratios

        @staticmethod
        @once
        def backward(ctx, grad_loss, _):
            logits, ids, stats = ctx.saved_tensors
            return (c.preference_loss_backward(logits, ids, stats, _contiguous(grad_loss), ctx.temperature),) + (None,) * 10

    _functions = Score, Policy, Preference
    return _functions


def score(logits, ids, temperature=1.0, entropy=False):
    """(log_probs, entropy) of tokens `ids` (float32 [n]; entropy None unless
    asked for) as an autograd function of the logits: token_log_probs forward,
    token_log_probs_backward backward."""
    return _autograd()[0].apply(logits, ids, temperature, entropy)


def policy(logits, ids, advantages, old_log_probs=None, ref_log_probs=None, weights=None, temperature=1.0, clip_low=0.2,
           clip_high=0.2, dual_clip=0.0, kl_coef=0.0, kl="k3", entropy_coef=0.0, entropy=False):
    """The policy loss per row (float32 [n]) and its metrics (float32 [n, 4], no
    gradient) as an autograd function of the logits: policy_loss forward,
    policy_loss_backward backward."""
    return _autograd()[1].apply(logits, ids, advantages, old_log_probs, ref_log_probs, weights, temperature, clip_low,
                                clip_high, dual_clip, kl_coef, kl, entropy_coef, entropy)


def preference(logits, ids, answer_offsets, ref_log_probs=None, weights=None, temperature=1.0, beta=0.1, loss="sigmoid",
               label_smoothing=0.0, margin=0.0, average=False):
    """The preference loss per pair (float32 [pairs]) and the answers' log-ratios
    (float32 [2 * pairs], no gradient) as an autograd function of the logits:
    preference_loss forward, preference_loss_backward backward."""
    return _autograd()[2].apply(logits, ids, answer_offsets, ref_log_probs, weights, temperature, beta, loss,
                                label_smoothing, margin, average)
