"""Python side of include/ls_row_ops.h: penalties, biases and masks before
sampling, top log-probs beside it, the distillation loss and its gradient.

The calls themselves (process_logits, top_log_probs, distill_loss,
distill_loss_backward, distill_loss_grad) are functions of the extension module
_row_ops_c (csrc/py/row_ops_py.cpp): argument checks and marshalling only.  They
are loaded, with torch, when the package's attribute of that name is first
used."""
import ctypes
import importlib.util
import os
from dataclasses import dataclass

from . import _binding, _token_ops
from ._binding import LSError, load_library

LS_ROW_ERR_BAD_MASK = 8
MAX_TOP = 256  # LS_MAX_TOP
DISTILL_STATS = 8  # LS_DISTILL_STATS
CALLS = ("process_logits", "top_log_probs", "distill_loss", "distill_loss_backward", "distill_loss_grad")

_P, _i32t, _i64t, _f32t, _ci = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_int


class _LogitsParams(ctypes.Structure):
    _fields_ = [("tokens", _P), ("token_stride", _i64t), ("token_capacity", _i32t), ("prompt_lens", _P),
                ("seq_lens", _P), ("repetition", _P), ("presence", _P), ("frequency", _P), ("bias_offsets", _P),
                ("bias_ids", _P), ("bias_values", _P), ("bias_count", _i32t), ("num_requests", _i32t)]


class _Field(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("tensor", ctypes.py_object), ("data", _P), ("numel", _i64t)]


class _Marshalled(ctypes.Structure):
    """What process_logits reads of a LogitsParams: the C struct, and the tensors as they were when it was made."""
    _fields_ = [("params", _LogitsParams), ("device", _i32t), ("count", _i32t), ("fields", _Field * 9)]


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
    lib.ls_set_process_policy.argtypes = [ci]
    lib.ls_set_process_policy.restype = ci
    lib.ls_row_ops_max_vocab.argtypes = [ci]
    lib.ls_row_ops_max_vocab.restype = i64
    return lib


_ready = None


def _lib():
    global _ready
    lib = load_library()
    if _ready is not lib:
        _ready = _token_ops.configure(configure(lib))
    return lib


def set_process_policy(policy):
    """ls_set_process_policy: 0 chosen from the batch, 1 one kernel, 2 a copying
    and a settling kernel (process_logits; every later call of the process)."""
    st = _lib().ls_set_process_policy(int(policy))
    if st != _binding.LS_OK:
        raise LSError(st, f"ls_set_process_policy({policy})")


_calls = None


def calls():
    """The extension module with the calls, bound to the loaded library (raises
    if either is missing)."""
    global _calls
    if _calls is None:
        lib = _lib()
        path = os.path.join(_binding.PKG, "_row_ops_c.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m logits_sampling_gb300.build` "
                               "(there is no CPU fallback)")
        from . import build
        if build.binding_built_for() != build.binding_target():
            raise RuntimeError(f"{path} was built for {build.binding_built_for() or 'an unknown torch'}, this is "
                               f"{build.binding_target()}: run `python -m logits_sampling_gb300.build`")
        import torch  # noqa: F401  (its libraries first: the module links against them)
        spec = importlib.util.spec_from_file_location("logits_sampling_gb300._row_ops_c", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(LSError, *(ctypes.cast(getattr(lib, "ls_" + name), ctypes.c_void_p).value
                               for name in CALLS + _token_ops.CALLS))
        _calls = module
    return _calls


def row_ops_max_vocab(dtype):
    """ls_row_ops_max_vocab: the largest vocab of top_log_probs and the distillation calls."""
    return int(_lib().ls_row_ops_max_vocab(int(dtype)))


def _vec(t, dtype, what):
    """The pointer of an optional contiguous device tensor."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {str(dtype)[6:]}")
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    return t.data_ptr()


@dataclass(frozen=True, eq=False)
class LogitsParams:
    """Per-request parameters of process_logits as device tensors, for R requests.

    tokens int32 [R, capacity] holds each request's ids, the prompt's first;
    seq_lens int32 [R] how many of them there are and prompt_lens int32 [R] how
    many belong to the prompt.  The caller appends to tokens and seq_lens as it
    samples.  Penalties are float32 [R].  Biases are a ragged list: request r
    owns bias_ids/bias_values[bias_offsets[r]:bias_offsets[r + 1]], ids distinct.
    Fields left None switch their part off.  Values may change in place at any
    time; a tensor that is resized or given another storage needs a new
    LogitsParams (the calls refuse the old one)."""
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
        kept = _Marshalled(params=self._marshal())
        fields = {name: t for name, t in vars(self).items() if t is not None}
        devices = {t.device for t in fields.values()}
        if len(devices) > 1:
            raise ValueError(f"fields lie on different devices: {sorted(map(str, devices))}")
        # the addresses are valid while the tensors keep their storages: the calls refuse one that does not
        kept.device, kept.count = devices.pop().index, len(fields)
        for field, (name, t) in zip(kept.fields, fields.items()):
            field.name, field.tensor, field.data, field.numel = name.encode(), t, t.data_ptr(), t.numel()
        object.__setattr__(self, "_kept", kept)
        object.__setattr__(self, "_marshalled", ctypes.addressof(kept))

    def _marshal(self):
        import torch

        def i32(t, what):
            return _vec(t, torch.int32, what)

        def f32(t, what):
            return _vec(t, torch.float32, what)

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
            s.bias_offsets = i32(self.bias_offsets, "bias_offsets")
            s.bias_ids = i32(self.bias_ids, "bias_ids")
            s.bias_values = f32(self.bias_values, "bias_values")
            s.bias_count = int(self.bias_ids.numel())
        if not counts:
            raise ValueError("LogitsParams needs tokens or biases")
        if len(set(counts.values())) > 1:
            raise ValueError(f"fields disagree on the number of requests: {counts}")
        s.num_requests = next(iter(counts.values()))
        s.prompt_lens = i32(self.prompt_lens, "prompt_lens")
        s.seq_lens = i32(self.seq_lens, "seq_lens")
        s.repetition = f32(self.repetition_penalty, "repetition_penalty")
        s.presence = f32(self.presence_penalty, "presence_penalty")
        s.frequency = f32(self.frequency_penalty, "frequency_penalty")
        return s

    @staticmethod
    def from_host(histories=None, prompt_lens=None, capacity=None, repetition_penalty=None, presence_penalty=None,
                  frequency_penalty=None, biases=None, device="cuda"):
        """Builds the tensors from host lists: `histories` a list of id lists
        (with room for `capacity` ids each), `biases` a list of {id: bias} dicts."""
        import numpy as np
        import torch

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


def distill(logits, teacher_ids, teacher_log_probs, temperature=1.0, tail="bucket", weights=None):
    """The distillation loss per row (float32 [n]) as an autograd function of
    the logits: distill_loss forward, distill_loss_backward backward."""
    global _Distill
    if _Distill is None:
        import torch
        c = calls()

        class Distill(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, ids, log_probs, temperature, tail, weights):
                loss, stats = c.distill_loss(logits, ids, log_probs, temperature, tail, weights)
                ctx.save_for_backward(logits, ids, log_probs, stats, weights)
                ctx.how = (temperature, tail)
                return loss

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, grad_loss):
                logits, ids, log_probs, stats, weights = ctx.saved_tensors
                temperature, tail = ctx.how
                return c.distill_loss_backward(logits, ids, log_probs, stats, grad_loss.float().contiguous(),
                                             temperature, tail, weights), None, None, None, None, None

        _Distill = Distill
    return _Distill.apply(logits, teacher_ids, teacher_log_probs, temperature, tail, weights)


_Distill = None
