"""ctypes binding of include/ls_row_ops.h (argument marshalling only): penalties,
biases and masks before sampling, top log-probs beside it, the distillation
loss and its gradient."""
import ctypes
import functools
from dataclasses import dataclass

from ._binding import LS_DTYPE_BF16, LS_DTYPE_F32, LS_OK, LSError, load_library

torch = None  # imported by the first call: building the library needs no torch
_DTYPES = {}

LS_ROW_ERR_BAD_MASK = 8
MAX_TOP = 256  # LS_MAX_TOP
DISTILL_STATS = 8  # LS_DISTILL_STATS
TAILS = {"drop": 0, "renorm": 1, "bucket": 2}

_P, _i32t, _i64t, _f32t, _ci = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_int


class _LogitsParams(ctypes.Structure):
    _fields_ = [("tokens", _P), ("token_stride", _i64t), ("token_capacity", _i32t), ("prompt_lens", _P),
                ("seq_lens", _P), ("repetition", _P), ("presence", _P), ("frequency", _P), ("bias_offsets", _P),
                ("bias_ids", _P), ("bias_values", _P), ("bias_count", _i32t), ("num_requests", _i32t)]


class _Teacher(ctypes.Structure):
    _fields_ = [("ids", _P), ("log_probs", _P), ("stride", _i64t), ("k", _i32t)]


def configure(lib):
    """Declare the C signatures of include/ls_row_ops.h on a loaded library."""
    P, i32, i64, f32, ci = _P, _i32t, _i64t, _f32t, _ci
    PP, PT = ctypes.POINTER(_LogitsParams), ctypes.POINTER(_Teacher)
    lib.ls_process_logits.argtypes = [P, ci, i64, i64, i64, i32, P, P, PP, P, P, i64, i64, P, P, i64, P, P]
    lib.ls_top_log_probs.argtypes = [P, ci, i64, i64, i64, i32, P, i32, f32, P, P, P, P, P]
    lib.ls_distill_loss.argtypes = [P, ci, i64, i64, i32, PT, f32, ci, P, P, P, P, P]
    lib.ls_distill_loss_backward.argtypes = [P, ci, i64, i64, i32, PT, f32, ci, P, P, P, P, i64, P]
    lib.ls_distill_loss_grad.argtypes = [P, ci, i64, i64, i32, PT, f32, ci, P, P, P, i64, P, P]
    for name in ("ls_process_logits", "ls_top_log_probs", "ls_distill_loss", "ls_distill_loss_backward",
                 "ls_distill_loss_grad"):
        getattr(lib, name).restype = ci
    lib.ls_row_ops_max_vocab.argtypes = [ci]
    lib.ls_row_ops_max_vocab.restype = i64
    return lib


_ready = None


def _need_torch():
    global torch
    if torch is None:
        import torch as t
        torch = t
        _DTYPES.update({t.float32: LS_DTYPE_F32, t.bfloat16: LS_DTYPE_BF16})


def _lib():
    global _ready
    lib = load_library()
    if _ready is not lib:
        _need_torch()
        _ready = configure(lib)
    return lib


def row_ops_max_vocab(dtype):
    """ls_row_ops_max_vocab: the largest vocab of top_log_probs and the distillation calls."""
    return int(_lib().ls_row_ops_max_vocab(int(dtype)))


def _matrix(logits):
    """(pointer, dtype, rows, vocab, row stride, raw current stream) of a logits matrix."""
    dt = _DTYPES.get(logits.dtype)
    if dt is None:
        raise TypeError(f"unsupported logits dtype {logits.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [rows, vocab]")
    stride, inner = logits.stride()
    if inner != 1:
        raise ValueError("logits rows must be contiguous (stride(1) == 1)")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    rows, vocab = logits.shape
    if rows <= 1 and stride < vocab:
        stride = vocab
    return logits.data_ptr(), dt, rows, vocab, stride, torch._C._cuda_getCurrentRawStream(logits.get_device())


def _on_stream(f):
    """A call's `stream` argument: the call runs with that stream current, so
    that its outputs are allocated on it.  Without one nothing is entered."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        _need_torch()
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


def _vec(t, dtype, what, n=None):
    """The pointer of a contiguous device tensor of at least n entries."""
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {str(dtype)[6:]}")
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    if n is not None and t.numel() < n:
        raise ValueError(f"{what} has {t.numel()} entries, {n} are needed")
    return t.data_ptr()


def _f32(t, what, n=None):
    return None if t is None else _vec(t, torch.float32, what, n)


def _i32(t, what, n=None):
    return None if t is None else _vec(t, torch.int32, what, n)


def _like(t, logits, n, what):
    """Checks a matrix of the logits' type that a call writes; its row stride."""
    if t.dtype != logits.dtype or t.dim() != 2 or t.shape[0] < n or t.shape[1] != logits.shape[1]:
        raise ValueError(f"{what} must be [{n}, {logits.shape[1]}] of {logits.dtype}")
    if t.stride(1) != 1:
        raise ValueError(f"{what}'s rows must be contiguous (stride(1) == 1)")
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


@dataclass(frozen=True, eq=False)
class LogitsParams:
    """Per-request parameters of process_logits as device tensors, for R requests.

    tokens int32 [R, capacity] holds each request's ids, the prompt's first;
    seq_lens int32 [R] how many of them there are and prompt_lens int32 [R] how
    many belong to the prompt.  The caller appends to tokens and seq_lens as it
    samples.  Penalties are float32 [R].  Biases are a ragged list: request r
    owns bias_ids/bias_values[bias_offsets[r]:bias_offsets[r + 1]], ids distinct.
    Fields left None switch their part off."""
    tokens: object = None
    prompt_lens: object = None
    seq_lens: object = None
    repetition_penalty: object = None
    presence_penalty: object = None
    frequency_penalty: object = None
    bias_offsets: object = None
    bias_ids: object = None
    bias_values: object = None

    def __post_init__(self):
        struct = self._marshal()  # its pointers stay valid with the tensors that the fields hold
        object.__setattr__(self, "_struct", struct)
        object.__setattr__(self, "_ref", ctypes.byref(struct))

    def _marshal(self):
        _need_torch()
        per_request = {"prompt_lens": self.prompt_lens, "seq_lens": self.seq_lens,
                       "repetition_penalty": self.repetition_penalty, "presence_penalty": self.presence_penalty,
                       "frequency_penalty": self.frequency_penalty}
        counts = {name: int(t.numel()) for name, t in per_request.items() if t is not None}
        s = _LogitsParams()
        if self.tokens is not None:
            if self.tokens.dim() != 2 or (self.tokens.shape[1] > 1 and self.tokens.stride(1) != 1):
                raise ValueError("tokens must be [requests, capacity] with contiguous rows")
            if self.tokens.dtype != torch.int32:
                raise TypeError("tokens must be int32")
            if not self.tokens.is_cuda:
                raise ValueError("expected a CUDA tensor")
            counts["tokens"] = int(self.tokens.shape[0])
            s.tokens = self.tokens.data_ptr()
            s.token_stride = self.tokens.stride(0) if self.tokens.shape[0] > 1 and self.tokens.numel() else self.tokens.shape[1]
            s.token_capacity = self.tokens.shape[1]
        if self.bias_offsets is not None:
            counts["bias_offsets"] = int(self.bias_offsets.numel()) - 1
            if self.bias_ids is None or self.bias_values is None or self.bias_ids.numel() != self.bias_values.numel():
                raise ValueError("bias_ids and bias_values must come with bias_offsets and be equally long")
            s.bias_offsets = _i32(self.bias_offsets, "bias_offsets")
            s.bias_ids = _i32(self.bias_ids, "bias_ids")
            s.bias_values = _f32(self.bias_values, "bias_values")
            s.bias_count = int(self.bias_ids.numel())
        if not counts:
            raise ValueError("LogitsParams needs tokens or biases")
        if len(set(counts.values())) > 1:
            raise ValueError(f"fields disagree on the number of requests: {counts}")
        s.num_requests = next(iter(counts.values()))
        s.prompt_lens = _i32(self.prompt_lens, "prompt_lens")
        s.seq_lens = _i32(self.seq_lens, "seq_lens")
        s.repetition = _f32(self.repetition_penalty, "repetition_penalty")
        s.presence = _f32(self.presence_penalty, "presence_penalty")
        s.frequency = _f32(self.frequency_penalty, "frequency_penalty")
        return s

    @staticmethod
    def from_host(histories=None, prompt_lens=None, capacity=None, repetition_penalty=None, presence_penalty=None,
                  frequency_penalty=None, biases=None, device="cuda"):
        """Builds the tensors from host lists: `histories` a list of id lists
        (with room for `capacity` ids each), `biases` a list of {id: bias} dicts."""
        import numpy as np

        def dev(v, dtype):
            return None if v is None else torch.from_numpy(np.ascontiguousarray(v, dtype)).to(device)

        tokens = seq = offsets = ids = values = None
        if histories is not None:
            seq = [len(h) for h in histories]
            cap = max(max(seq, default=0), capacity or 0, 1)
            tokens = np.full((len(histories), cap), -1, np.int32)
            for row, h in zip(tokens, histories):
                row[:len(h)] = h
            if prompt_lens is None:
                prompt_lens = seq
        if biases is not None:
            offsets = np.cumsum([0] + [len(b) for b in biases])
            ids = [j for b in biases for j in b.keys()]
            values = [v for b in biases for v in b.values()]
        return LogitsParams(dev(tokens, np.int32), dev(prompt_lens, np.int32), dev(seq, np.int32),
                            dev(repetition_penalty, np.float32), dev(presence_penalty, np.float32),
                            dev(frequency_penalty, np.float32), dev(offsets, np.int32), dev(ids, np.int32),
                            dev(values, np.float32))


@_on_stream
def process_logits(logits, n=None, params=None, gather_indices=None, token_to_request_index=None, row_lens=None,
                   allowed_mask=None, mask_index=None, out=None, error_word=None):
    """ls_process_logits: returns out ([n, vocab] of the logits' type).  out may
    be the logits themselves (no gather_indices).  allowed_mask int32
    [mask_rows, >= ceil(vocab / 32)].  `stream`: the current one by default."""
    lib = _ready or _lib()
    ptr, dt, rows, V, stride, raw = _matrix(logits)
    if n is None:
        n = len(gather_indices) if gather_indices is not None else rows
    mask_ptr, mask_rows, mask_stride = None, 0, 0
    if allowed_mask is not None:
        if allowed_mask.dim() != 2 or allowed_mask.stride(1) != 1 or allowed_mask.dtype is not torch.int32:
            raise ValueError("allowed_mask must be int32 [mask_rows, words] with contiguous rows")
        if not allowed_mask.is_cuda:
            raise ValueError("expected a CUDA tensor")
        mask_ptr, (mask_rows, words) = allowed_mask.data_ptr(), allowed_mask.shape
        mask_stride = allowed_mask.stride(0) if mask_rows > 1 else words
    if out is None:
        out = torch.empty((n, V), dtype=logits.dtype, device=logits.device)
        out_stride = V
    else:
        out_stride = _like(out, logits, n, "out")
    st = lib.ls_process_logits(
        ptr, dt, rows, V, stride, n, _i32(gather_indices, "gather_indices", n),
        _i32(token_to_request_index, "token_to_request_index", n), None if params is None else params._ref,
        _i32(row_lens, "row_lens", n), mask_ptr, mask_rows, mask_stride, _i32(mask_index, "mask_index", n),
        out.data_ptr(), out_stride, _i32(error_word, "error_word"), raw)
    if st != LS_OK:
        raise LSError(st, "ls_process_logits")
    return out


@_on_stream
def top_log_probs(logits, k, n=None, temperature=1.0, gather_indices=None, out_ids=None, out_log_probs=None,
                  out_lse=None, error_word=None):
    """ls_top_log_probs: returns (ids int32 [n, k], log_probs float32 [n, k], lse
    float32 [n]).  `stream`: the current one by default."""
    lib = _ready or _lib()
    ptr, dt, rows, V, stride, raw = _matrix(logits)
    if n is None:
        n = len(gather_indices) if gather_indices is not None else rows
    dev = logits.device
    if out_ids is None:
        out_ids = torch.empty((n, k), dtype=torch.int32, device=dev)
    else:
        _i32(out_ids, "out_ids", n * k)
    if out_log_probs is None:
        out_log_probs = torch.empty((n, k), dtype=torch.float32, device=dev)
    else:
        _f32(out_log_probs, "out_log_probs", n * k)
    if out_lse is None:
        out_lse = torch.empty(n, dtype=torch.float32, device=dev)
    else:
        _f32(out_lse, "out_lse", n)
    st = lib.ls_top_log_probs(ptr, dt, rows, V, stride, n, _i32(gather_indices, "gather_indices", n), k, temperature,
                              out_ids.data_ptr(), out_log_probs.data_ptr(), out_lse.data_ptr(),
                              _i32(error_word, "error_word"), raw)
    if st != LS_OK:
        raise LSError(st, f"ls_top_log_probs (k = {k}; at most {MAX_TOP})")
    return out_ids, out_log_probs, out_lse


def _teacher(ids, log_probs, n):
    k = ids.shape[-1]
    if ids.shape != (n, k) or log_probs.shape != (n, k):
        raise ValueError(f"teacher_ids and teacher_log_probs must both be [{n}, k]")
    if ids.dtype is not torch.int32 or log_probs.dtype is not torch.float32:
        raise TypeError("teacher_ids must be int32, teacher_log_probs float32")
    stride, inner = ids.stride()
    if n <= 1:
        stride = k
    elif log_probs.stride(0) != stride:
        raise ValueError("teacher_ids and teacher_log_probs must have one row stride")
    if k > 1 and (inner != 1 or log_probs.stride(1) != 1):
        raise ValueError("teacher_ids and teacher_log_probs must have contiguous rows")
    if not (ids.is_cuda and log_probs.is_cuda):
        raise ValueError("expected a CUDA tensor")
    return ctypes.byref(_Teacher(ids.data_ptr(), log_probs.data_ptr(), stride, k))


def _tail(tail):
    code = TAILS.get(tail)
    if code is None:
        raise ValueError(f"tail must be one of {sorted(TAILS)}")
    return code


@_on_stream
def distill_loss(logits, teacher_ids, teacher_log_probs, temperature=1.0, tail="bucket", weights=None, out=None,
                 out_stats=None, error_word=None):
    """ls_distill_loss: returns (loss float32 [n], stats float32 [n, 8]); stats
    goes to distill_loss_backward.  `stream`: the current one by default."""
    lib = _ready or _lib()
    ptr, dt, n, V, stride, raw = _matrix(logits)
    teacher = _teacher(teacher_ids, teacher_log_probs, n)
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=logits.device)
    else:
        _f32(out, "out", n)
    if out_stats is None:
        out_stats = torch.empty((n, DISTILL_STATS), dtype=torch.float32, device=logits.device)
    else:
        _f32(out_stats, "out_stats", DISTILL_STATS * n)
    st = lib.ls_distill_loss(ptr, dt, V, stride, n, teacher, temperature, _tail(tail), _f32(weights, "weights", n),
                             out.data_ptr(), out_stats.data_ptr(), _i32(error_word, "error_word"), raw)
    if st != LS_OK:
        raise LSError(st, "ls_distill_loss")
    return out, out_stats


@_on_stream
def distill_loss_backward(logits, teacher_ids, teacher_log_probs, stats, grad_loss=None, temperature=1.0,
                          tail="bucket", weights=None, out=None):
    """ls_distill_loss_backward: returns out, the gradient ([n, vocab] of the
    logits' type; out may be the logits themselves).  `stream`: the current one
    by default."""
    lib = _ready or _lib()
    ptr, dt, n, V, stride, raw = _matrix(logits)
    teacher = _teacher(teacher_ids, teacher_log_probs, n)
    if out is None:
        out = torch.empty((n, V), dtype=logits.dtype, device=logits.device)
        out_stride = V
    else:
        out_stride = _like(out, logits, n, "out")
    st = lib.ls_distill_loss_backward(ptr, dt, V, stride, n, teacher, temperature, _tail(tail),
                                      _f32(weights, "weights", n), _f32(stats, "stats", DISTILL_STATS * n),
                                      _f32(grad_loss, "grad_loss", n), out.data_ptr(), out_stride, raw)
    if st != LS_OK:
        raise LSError(st, "ls_distill_loss_backward")
    return out


@_on_stream
def distill_loss_grad(logits, teacher_ids, teacher_log_probs, temperature=1.0, tail="bucket", weights=None,
                      out_loss=None, out_grad=None, error_word=None):
    """ls_distill_loss_grad: returns (loss float32 [n], gradient [n, vocab] of
    the logits' type) from one call; out_grad may be the logits themselves.
    `stream`: the current one by default."""
    lib = _ready or _lib()
    ptr, dt, n, V, stride, raw = _matrix(logits)
    teacher = _teacher(teacher_ids, teacher_log_probs, n)
    if out_loss is None:
        out_loss = torch.empty(n, dtype=torch.float32, device=logits.device)
    else:
        _f32(out_loss, "out_loss", n)
    if out_grad is None:
        out_grad = torch.empty((n, V), dtype=logits.dtype, device=logits.device)
        out_stride = V
    else:
        out_stride = _like(out_grad, logits, n, "out_grad")
    st = lib.ls_distill_loss_grad(ptr, dt, V, stride, n, teacher, temperature, _tail(tail),
                                  _f32(weights, "weights", n), out_loss.data_ptr(), out_grad.data_ptr(), out_stride,
                                  _i32(error_word, "error_word"), raw)
    if st != LS_OK:
        raise LSError(st, "ls_distill_loss_grad")
    return out_loss, out_grad


def distill(logits, teacher_ids, teacher_log_probs, temperature=1.0, tail="bucket", weights=None):
    """The distillation loss per row (float32 [n]) as an autograd function of
    the logits: distill_loss forward, distill_loss_backward backward."""
    global _Distill
    if _Distill is None:
        _need_torch()

        class Distill(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, ids, log_probs, temperature, tail, weights):
                loss, stats = distill_loss(logits, ids, log_probs, temperature, tail, weights)
                ctx.save_for_backward(logits, ids, log_probs, stats, weights)
                ctx.how = (temperature, tail)
                return loss

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, grad_loss):
                logits, ids, log_probs, stats, weights = ctx.saved_tensors
                temperature, tail = ctx.how
                return distill_loss_backward(logits, ids, log_probs, stats, grad_loss.float().contiguous(),
                                             temperature, tail, weights), None, None, None, None, None

        _Distill = Distill
    return _Distill.apply(logits, teacher_ids, teacher_log_probs, temperature, tail, weights)


_Distill = None
