"""Binding of the logit operators around the verify step (C ABI in
``include/sd_logits.h``): token counts, penalties with biases and grammar
masks, a teacher's top logits, and the distillation loss with its gradient.

Like the rest of the package this module only checks and marshals arguments.
Memory that the caller hands over to be written (out, counts, grad) counts as
changed in place for autograd: a backward pass that still needs what an
operation saved of it raises torch's error instead of reading other values.

  token_counts(...), token_counts_add(...)   sd_token_counts, sd_token_counts_add
  process_logits(...)                        sd_process_logits
  top_logits(...)                            sd_top_logits
  distill_loss(...), distill_grad(...)       sd_distill
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _P, SD_BF16, SD_F32, _check, _need, _on_stream, lib

SD_STATUS_BAD_PENALTY = 0x8
SD_MAX_TOP, SD_MAX_BIAS = 128, 1024

_DTYPES = {torch.float32: SD_F32, torch.bfloat16: SD_BF16}


class ProcessArgs(ctypes.Structure):
    """Mirror of ``sd_process_args`` in include/sd_logits.h."""
    _fields_ = [
        ("B", ctypes.c_int32), ("R", ctypes.c_int32), ("V", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("logits", _P), ("logits_sb", ctypes.c_int64),
        ("logits_sr", ctypes.c_int64), ("out", _P), ("out_sb", ctypes.c_int64),
        ("out_sr", ctypes.c_int64), ("counts", _P), ("prev", _P), ("P", ctypes.c_int32),
        ("base", ctypes.c_int32), ("repetition", _P), ("presence", _P), ("frequency", _P),
        ("bias_ids", _P), ("bias_vals", _P), ("n_bias", ctypes.c_int32), ("mask", _P),
        ("mask_sb", ctypes.c_int64), ("mask_sr", ctypes.c_int64), ("status", _P),
    ]


class DistillArgs(ctypes.Structure):
    """Mirror of ``sd_distill_args`` in include/sd_logits.h."""
    _fields_ = [
        ("N", ctypes.c_int32), ("V", ctypes.c_int32), ("k", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("student", _P), ("student_s", ctypes.c_int64), ("ids", _P),
        ("vals", _P), ("rest", _P), ("weight", _P), ("T", ctypes.c_float), ("loss", _P),
        ("grad", _P), ("grad_s", ctypes.c_int64), ("status", _P),
    ]


class TopLogits(NamedTuple):
    vals: torch.Tensor   # [...][k] float32, larger first
    ids: torch.Tensor    # [...][k] int32, -1 where nothing is left
    rest: torch.Tensor   # [...] float32: log sum exp(x / T) of the others


def _bind(L):
    """Argument types of the entry points, and the structs' layouts."""
    i32, i64, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    L.sd_token_counts.argtypes = [i32, i32, i32, _P, _P, _P, _P, _P, _P]
    L.sd_token_counts_add.argtypes = [i32, i32, i32, _P, _P, _P, _P, _P]
    L.sd_process_logits.argtypes = [ctypes.POINTER(ProcessArgs), _P]
    L.sd_top_logits.argtypes = [i32, i32, i32, _P, i64, i32, f32, _P, _P, _P, _P]
    L.sd_distill.argtypes = [ctypes.POINTER(DistillArgs), _P]
    for fn in (L.sd_token_counts, L.sd_token_counts_add, L.sd_process_logits, L.sd_top_logits,
               L.sd_distill):
        fn.restype = ctypes.c_int
    for fn, mirror in ((L.sd_process_args_size, ProcessArgs),
                       (L.sd_distill_args_size, DistillArgs)):
        fn.argtypes, fn.restype = [], ctypes.c_size_t
        if fn() != ctypes.sizeof(mirror):
            raise RuntimeError(f"{mirror.__name__} layout differs between library and binding")


# the current stream's handle by device index, without making a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_written = torch.autograd.graph.increment_version   # of a tensor of the caller's

_loaded = None   # the library, once a call has needed it


def _lib():
    global _loaded
    if _loaded is None:
        _loaded = lib()
    return _loaded


def _stream_of(device):
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _rows(t, name, dims):
    """Checks a tensor of logit rows: CUDA, float32 or bfloat16, each row contiguous."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.dim() not in dims:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected {' or '.join(map(str, dims))}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return dt


def _arg(t, name, dtype, shape, device):
    """The address of a required array; what is wrong with it is said by _need."""
    if t is None or t.dtype is not dtype or t.device != device or t.shape != shape \
            or not t.is_contiguous():
        _need(t, name, dtype, shape, device)
    return t.data_ptr()


def _same(x, out):
    """Whether two tensors of one shape are the same memory, element by element (the stride
    of a dimension of one says nothing)."""
    return x.data_ptr() == out.data_ptr() and all(
        a == b for n, a, b in zip(x.shape, x.stride(), out.stride()) if n > 1)


def _apart(x, out):
    """Whether the ranges of addresses of two tensors are disjoint."""
    ends = lambda t: t.data_ptr() + t.element_size() * (
        1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))
    return not x.numel() or out.data_ptr() >= ends(x) or x.data_ptr() >= ends(out)


def _overlap(x, out):
    """Whether two tensors of contiguous rows, of one shape and type, share an element: rows
    of one may lie between those of the other."""
    if _apart(x, out):
        return False

    def starts(t):   # the rows' addresses, in order
        a = torch.tensor(t.data_ptr(), device="cpu")
        for n, s in zip(t.shape[:-1], t.stride()[:-1]):
            a = a[..., None] + torch.arange(n, device="cpu") * (s * t.element_size())
        return a.flatten().sort().values

    # a row meets one of the other tensor's only if it meets the next one up or down
    a, b, size = starts(x), starts(out), x.shape[-1] * x.element_size()
    up = torch.searchsorted(b, a)
    above, below = b[up.clamp(max=len(b) - 1)], b[(up - 1).clamp(min=0)]
    return bool(((above - a).abs() < size).any() or ((a - below).abs() < size).any())


def _out_like(x, out, name):
    """Checks an output given by the caller: shape and type of x, rows contiguous,
    either x itself or memory of its own."""
    _rows(out, name, (x.dim(),))
    if out.dtype != x.dtype or out.shape != x.shape or out.device != x.device:
        raise ValueError(f"{name} must have the shape, type and device of the input")
    if not _same(x, out) and _overlap(x, out):
        raise ValueError(f"{name} overlaps the input without being the same tensor")


@_on_stream
def token_counts(history, lengths, V: int, *, prompt_lengths=None, out=None, status=None,
                 stream=None) -> torch.Tensor:
    """counts [B][V] int16 of history [B][L] (int32), lengths [B] and
    prompt_lengths [B] (int32, none: no prompt): the low 15 bits are how often
    the output text holds the token (at most 32767), the sign bit is set where
    the prompt holds it."""
    _need(history, "history", torch.int32)
    if history.dim() != 2:
        raise ValueError("history must be [B][L]")
    B, L = history.shape
    dev = history.device
    _need(lengths, "lengths", torch.int32, (B,), dev)
    given = out is not None
    if given:
        _need(out, "out", torch.int16, (B, V), dev)
    else:
        out = torch.empty((B, V), dtype=torch.int16, device=dev)
    prompt = st = None
    if prompt_lengths is not None:
        prompt = _arg(prompt_lengths, "prompt_lengths", torch.int32, (B,), dev)
    if status is not None:
        st = _arg(status, "status", torch.int32, (1,), dev)
    _check(_lib().sd_token_counts(B, L, V, history.data_ptr(), lengths.data_ptr(), prompt,
                                  out.data_ptr(), st, _stream_of(dev)), "sd_token_counts")
    if given:
        _written(out)
    return out


@_on_stream
def token_counts_add(counts, tokens, n, *, status=None, stream=None) -> torch.Tensor:
    """Adds tokens[b][:n[b]] of tokens [B][M] to counts [B][V] in place: after a
    round, out_tokens and tau of its VerifyResult."""
    _need(counts, "counts", torch.int16)
    if counts.dim() != 2:
        raise ValueError("counts must be [B][V]")
    B, V = counts.shape
    dev = counts.device
    _need(tokens, "tokens", torch.int32, None, dev)
    if tokens.dim() != 2 or tokens.shape[0] != B:
        raise ValueError("tokens must be [B][M]")
    _need(n, "n", torch.int32, (B,), dev)
    st = None if status is None else _arg(status, "status", torch.int32, (1,), dev)
    _check(_lib().sd_token_counts_add(B, tokens.shape[1], V, tokens.data_ptr(), n.data_ptr(),
                                      counts.data_ptr(), st, _stream_of(dev)),
           "sd_token_counts_add")
    _written(counts)
    return counts


@_on_stream
def process_logits(logits, *, counts=None, prev=None, base: int = 0, repetition=None,
                   presence=None, frequency=None, bias_ids=None, bias_vals=None, mask=None,
                   out=None, status=None, stream=None) -> torch.Tensor:
    """Logits [B][R][V] (or [B][V]: one row each) under penalties, biases and a
    grammar's mask, as the verify step should see them.

    counts [B][V] int16 (token_counts); prev [B][P] int32: this round's drafts,
    of which row r counts prev[b][:base + r] (target rows of a round: the
    drafted tokens and base 0); repetition, presence, frequency [B] float32;
    bias_ids [B][n] int32 (-1: empty) with bias_vals [B][n] float32; mask
    [B][R][ceil(V / 32)] or [B][ceil(V / 32)] int32, a set bit allows the
    token.  All are optional.  out may be the logits tensor itself; there is no
    gradient of this step, so logits that are to be trained keep to an output
    of their own."""
    dt = _rows(logits, "logits", (2, 3))
    dev, shape = logits.device, logits.shape
    B, V = shape[0], shape[-1]
    R = shape[1] if len(shape) == 3 else 1
    given = out is not None
    if given:
        _out_like(logits, out, "out")
    else:
        out = torch.empty(shape, dtype=logits.dtype, device=dev)
    xs, ys = logits.stride(), out.stride()
    a = ProcessArgs(B, R, V, dt, logits.data_ptr(), xs[0], xs[1] if len(xs) == 3 else 0,
                    out.data_ptr(), ys[0], ys[1] if len(ys) == 3 else 0)
    if counts is not None:
        a.counts = _arg(counts, "counts", torch.int16, (B, V), dev)
    if prev is not None:
        if prev.dim() != 2:
            raise ValueError("prev must be [B][P]")
        P = prev.shape[1]
        if P == 0 and base + R > 1 and B and R:   # has no address: not given, to the library
            raise ValueError("prev must hold the base + R - 1 drafts that the rows count")
        a.prev, a.P, a.base = _arg(prev, "prev", torch.int32, (B, P), dev), P, base
    if repetition is not None:
        a.repetition = _arg(repetition, "repetition", torch.float32, (B,), dev)
    if presence is not None:
        a.presence = _arg(presence, "presence", torch.float32, (B,), dev)
    if frequency is not None:
        a.frequency = _arg(frequency, "frequency", torch.float32, (B,), dev)
    if bias_ids is not None:
        if bias_vals is None or bias_ids.dim() != 2:
            raise ValueError("bias_ids must be [B][n], with bias_vals")
        n = bias_ids.shape[1]
        ids = _arg(bias_ids, "bias_ids", torch.int32, (B, n), dev)
        vals = _arg(bias_vals, "bias_vals", torch.float32, (B, n), dev)
        if n:
            a.bias_ids, a.bias_vals, a.n_bias = ids, vals, n
    elif bias_vals is not None:
        raise ValueError("bias_vals needs bias_ids")
    if mask is not None:
        if not mask.is_cuda or mask.device != dev or mask.dtype != torch.int32:
            raise ValueError(f"mask must be an int32 tensor on {dev}")
        W = (V + 31) // 32
        ms = mask.stride()
        if mask.shape == (B, R, W):
            a.mask_sb, a.mask_sr = ms[0], ms[1]
        elif mask.shape == (B, W):
            a.mask_sb = ms[0]
        else:
            raise ValueError(f"mask has shape {tuple(mask.shape)}, expected {(B, R, W)} "
                             f"or {(B, W)}")
        if W > 1 and ms[-1] != 1:
            raise ValueError("mask must have contiguous rows")
        a.mask = mask.data_ptr()
    if status is not None:
        a.status = _arg(status, "status", torch.int32, (1,), dev)
    _check(_lib().sd_process_logits(a, _stream_of(dev)), "sd_process_logits")
    if given:
        _written(out)
    return out


def _row_stride(t, name):
    """Rows of a [N][V] or [A][B][V] tensor at one stride: (N, stride)."""
    if t.dim() == 2:
        return t.shape[0], t.stride(0)
    A, B, _ = t.shape
    if A > 1 and B > 1 and t.stride(0) != B * t.stride(1):
        raise ValueError(f"{name} must have its rows at one stride")
    return A * B, t.stride(1) if B > 1 else t.stride(0)


@_on_stream
def top_logits(logits, k: int, *, temperature: float = 1.0, out: TopLogits | None = None,
               stream=None) -> TopLogits:
    """The k largest logits of each row of [N][V] or [A][B][V] (ties to the
    lowest index, -inf never chosen) and the log-sum-exp at `temperature` of
    the others: what distill_loss and distill_grad take of a teacher."""
    dt = _rows(logits, "logits", (2, 3))
    dev, shape = logits.device, logits.shape
    N, stride = _row_stride(logits, "logits")
    lead = shape[:-1]
    kept = (*lead, k)
    given = out is not None
    if not given:
        out = TopLogits(torch.empty(kept, dtype=torch.float32, device=dev),
                        torch.empty(kept, dtype=torch.int32, device=dev),
                        torch.empty(lead, dtype=torch.float32, device=dev))
    else:
        _need(out.vals, "out.vals", torch.float32, kept, dev)
        _need(out.ids, "out.ids", torch.int32, kept, dev)
        _need(out.rest, "out.rest", torch.float32, lead, dev)
    _check(_lib().sd_top_logits(N, shape[-1], dt, logits.data_ptr(), stride, k, temperature,
                                out.vals.data_ptr(), out.ids.data_ptr(), out.rest.data_ptr(),
                                _stream_of(dev)), "sd_top_logits")
    if given:
        for t in out:
            _written(t)
    return out


def _distill(student, ids, vals, rest, temperature, weight, status, loss, grad):
    """sd_distill; loss and grad are checked where the caller gave them."""
    dt = _rows(student, "student", (2, 3))
    dev, shape = student.device, student.shape
    N, stride = _row_stride(student, "student")
    lead = shape[:-1]
    if ids.dim() != len(shape):
        raise ValueError("ids must have the student's leading dimensions and k")
    k = ids.shape[-1]
    kept = (*lead, k)
    a = DistillArgs(N, shape[-1], k, dt, student.data_ptr(), stride,
                    _arg(ids, "ids", torch.int32, kept, dev),
                    _arg(vals, "vals", torch.float32, kept, dev))
    if rest is not None:
        a.rest = _arg(rest, "rest", torch.float32, lead, dev)
    if weight is not None:
        a.weight = _arg(weight, "weight", torch.float32, lead, dev)
    a.T = temperature
    a.loss = loss.data_ptr()
    if grad is not None:
        a.grad, a.grad_s = grad.data_ptr(), _row_stride(grad, "grad")[1]
    if status is not None:
        a.status = _arg(status, "status", torch.int32, (1,), dev)
    _check(_lib().sd_distill(a, _stream_of(dev)), "sd_distill")


@_on_stream
def distill_loss(student, ids, vals, rest=None, *, temperature: float = 1.0, weight=None,
                 out=None, status=None, stream=None) -> torch.Tensor:
    """Distillation loss of each row of the student's logits ([N][V] or
    [A][B][V]) against a teacher's top logits (ids, vals, rest of top_logits at
    the same temperature; without rest the named tokens hold all of the
    teacher's mass): weight times the divergence of the k named tokens and one
    bucket of all others.  Evaluation: reads the logits once."""
    lead = student.shape[:-1]
    given = out is not None
    if given:
        _need(out, "out", torch.float32, lead, student.device)
    else:
        out = torch.empty(lead, dtype=torch.float32, device=student.device)
    _distill(student, ids, vals, rest, temperature, weight, status, out, None)
    if given:
        _written(out)
    return out


@_on_stream
def distill_grad(student, ids, vals, rest=None, *, temperature: float = 1.0, weight=None,
                 grad=None, status=None, stream=None):
    """(loss, grad): the loss of distill_loss and, in the same call, its gradient
    with respect to the student's logits, times `weight` (what reaches each
    row's loss from above: 1 / N for a mean).  To train: student.backward(grad).
    grad may be the student tensor itself where no operation saved it for its
    backward pass (a matrix product does not save its result, a tanh or softmax
    does, and so does a logsumexp of the same logits): that pass then raises."""
    loss = torch.empty(student.shape[:-1], dtype=torch.float32, device=student.device)
    given = grad is not None
    if not given:
        grad = torch.empty(student.shape, dtype=student.dtype, device=student.device)
    elif grad is not student:
        _out_like(student, grad, "grad")
    _distill(student, ids, vals, rest, temperature, weight, status, loss, grad)
    if given:
        _written(grad)
    return loss, grad
