"""GB300 token sampler: thin Python binding of libls_sampler.so.

The binding only marshals arguments (torch tensors -> device pointers, the
current CUDA stream) and calls the C ABI declared in include/ls_sampler.h:
``ls_sample``, ``ls_sample_speculative``, ``ls_log_probs``,
``ls_sample_log_probs``, ``ls_sample_log_probs_noalloc``, ``ls_sample_device_step``,
``ls_argmax``, ``ls_verify_chain``, ``ls_sample_verify``, ``ls_set_split_policy`` and
``ls_set_log_prob_write_policy``, and those of include/ls_row_ops.h around the
sampler: ``ls_process_logits``, ``ls_top_log_probs``, ``ls_distill_loss``,
``ls_distill_loss_backward`` and ``ls_distill_loss_grad``, and those of
include/ls_token_ops.h for training on sampled tokens: ``ls_token_log_probs``,
``ls_policy_loss`` and ``ls_preference_loss`` with their backward calls, and
``ls_policy_loss_grad``.  Every step of the sampling path runs in the library's
CUDA kernels; there is no CPU fallback.
If the library has not been built (``python -m logits_sampling_gb300.build``)
or no CUDA device is present, the calls raise.
"""
from ._binding import (  # noqa: F401
    LS_DTYPE_BF16,
    LS_DTYPE_F32,
    LS_ROW_ERR_BAD_GATHER,
    LS_ROW_ERR_BAD_REQUEST,
    LS_ROW_ERR_NO_FINITE,
    NOALLOC_MAX_ROWS,
    LSError,
    SamplingParams,
    argmax,
    lib_path,
    load_library,
    log_probs,
    max_vocab,
    sample,
    sample_device_step,
    sample_log_probs,
    sample_log_probs_noalloc,
    sample_speculative,
    sample_verify,
    set_log_prob_write_policy,
    set_split_policy,
    status_string,
    verify_chain,
)
from ._row_ops import (  # noqa: F401
    LS_ROW_ERR_BAD_MASK,
    MAX_TOP,
    LogitsParams,
    distill,
    row_ops_max_vocab,
    set_process_policy,
)
from ._token_ops import (  # noqa: F401
    LS_ROW_ERR_BAD_OFFSETS,
    POLICY_METRICS,
    TOKEN_STATS,
    policy,
    preference,
    score,
)


def __getattr__(name):
    """The calls of include/ls_row_ops.h and ls_token_ops.h, loaded (with torch) when first used."""
    from . import _row_ops, _token_ops
    if name in _row_ops.CALLS + _token_ops.CALLS:
        for call in _row_ops.CALLS + _token_ops.CALLS:
            globals()[call] = getattr(_row_ops.calls(), call)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
