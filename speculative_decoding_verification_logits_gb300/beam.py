"""Binding of beam search's step (C ABI in ``include/sd_beam.h``): the selection of the next beams
over beams and vocabulary, and the reordering of what a loop keeps per beam.  Paged caches
follow the same parents by kv_fork.

Like the rest of the package this module only checks and marshals arguments; every call takes
stream= as well, and runs on the current stream without it.

  beam_select(...)     sd_beam_select
  beam_reorder(...)    sd_beam_reorder
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import _P, _check, _need
from .kv import _all_apart, _i32, _lie_apart, _on_device, _rows_meet, _scratch, _small
from .logits import _lib, _rows, _same, _stream_of, _written

SD_MAX_BEAMS, SD_MAX_STATES = 32, 16


class SelectArgs(ctypes.Structure):
    """Mirror of ``sd_beam_select_args`` in include/sd_beam.h."""
    _fields_ = [
        *((n, ctypes.c_int32) for n in ("B", "W", "V", "k", "dtype")), ("logits", _P),
        ("logits_sb", ctypes.c_int64), ("logits_sw", ctypes.c_int64), ("scores", _P),
        ("finished", _P), ("norm", _P), ("eos", ctypes.c_int32), ("T", ctypes.c_float),
        ("out_scores", _P), ("parents", _P), ("tokens", _P), ("ended", _P), ("status", _P),
        ("workspace", _P), ("workspace_bytes", ctypes.c_size_t),
    ]


class StateArgs(ctypes.Structure):
    """Mirror of ``sd_beam_state`` in include/sd_beam.h."""
    _fields_ = [
        ("in_", _P), ("in_sb", ctypes.c_int64), ("in_sw", ctypes.c_int64), ("out", _P),
        ("out_sb", ctypes.c_int64), ("out_sw", ctypes.c_int64), ("row_bytes", ctypes.c_int64),
    ]


class Beams(NamedTuple):
    scores: torch.Tensor     # [B][k] float32, best first by score (over norm)
    parents: torch.Tensor    # [B][k] int32: the beam that each goes on from, -1: none
    tokens: torch.Tensor     # [B][k] int32, -1: none
    finished: torch.Tensor   # [B][k] uint8


def _bind(L):
    """Argument types of the entry points, and the structs' layouts."""
    i32, sz = ctypes.c_int32, ctypes.c_size_t
    L.sd_beam_select.argtypes = [ctypes.POINTER(SelectArgs), _P]
    L.sd_beam_reorder.argtypes = [i32, i32, i32, _P, i32, _P, _P, _P]
    L.sd_beam_select.restype = L.sd_beam_reorder.restype = ctypes.c_int
    L.sd_beam_select_workspace_size.argtypes = [i32, i32, i32, i32]
    L.sd_beam_select_workspace_size.restype = sz
    for fn, mirror in ((L.sd_beam_select_args_size, SelectArgs), (L.sd_beam_state_size, StateArgs)):
        fn.argtypes, fn.restype = [], sz
        if fn() != ctypes.sizeof(mirror):
            raise RuntimeError(f"{mirror.__name__} layout differs between library and binding")


@_on_device
def beam_select(logits, scores, k: int, *, temperature: float = 1.0, finished=None, eos: int = -1,
                norm=None, out: Beams | None = None, status=None) -> Beams:
    """The k best continuations of each sequence's beams: of scores [B][W] (float32, -inf: a
    beam that is dead) plus the log-softmax at `temperature` of logits [B][W][V] (float32 or
    bfloat16, contiguous rows), ranked by their score over norm [B][W] (float32, optional), ties
    to the lowest beam, then token.  finished [B][W] (uint8, with eos): such a beam stays as it is,
    with the token eos; a beam that emits eos is finished.  Slots left over hold -inf, -1, -1, 0."""
    dt = _rows(logits, "logits", (3,))
    dev = logits.device
    B, W, V = logits.shape
    _small(k, eos)
    a = SelectArgs(B, W, V, k, dt, logits.data_ptr(), logits.stride(0), logits.stride(1))
    if scores.dtype is not torch.float32 or scores.device != dev or scores.shape != (B, W) \
            or not scores.is_contiguous():
        _need(scores, "scores", torch.float32, (B, W), dev)
    a.scores, a.eos, a.T = scores.data_ptr(), eos, temperature
    if finished is not None:
        _need(finished, "finished", torch.uint8, (B, W), dev)
        if B:
            a.finished = finished.data_ptr()
    if norm is not None:
        _need(norm, "norm", torch.float32, (B, W), dev)
        a.norm = norm.data_ptr()
    if status is not None:
        a.status = _i32(status, "status", (1,), dev)
    n = _scratch("sd_beam_select_workspace_size", dev.index, B, W, V, dt) if B else 0
    ws = torch.empty(n, dtype=torch.int32, device=dev)
    given = ()
    if out is None:
        out = Beams(torch.empty((B, k), dtype=torch.float32, device=dev),
                    torch.empty((B, k), dtype=torch.int32, device=dev),
                    torch.empty((B, k), dtype=torch.int32, device=dev),
                    torch.empty((B, k), dtype=torch.uint8, device=dev))
        a.parents, a.tokens = out.parents.data_ptr(), out.tokens.data_ptr()
    else:
        _need(out.scores, "out.scores", torch.float32, (B, k), dev)
        _need(out.finished, "out.finished", torch.uint8, (B, k), dev)
        a.parents = _i32(out.parents, "out.parents", (B, k), dev)
        a.tokens = _i32(out.tokens, "out.tokens", (B, k), dev)
        given = out
        _all_apart(out, scores, finished, norm, status)
        if any(_rows_meet(logits, t.view(1, 1, B * k), 2) for t in out):
            raise ValueError("out overlaps the input")
    a.out_scores, a.ended = out.scores.data_ptr(), out.finished.data_ptr()
    a.workspace, a.workspace_bytes = ws.data_ptr(), 4 * n
    rc = _lib().sd_beam_select(a, _stream_of(dev))
    if rc:
        _check(rc, "sd_beam_select")
    for t in given:
        _written(t)
    return out


def _state(x, name, B, W, dev):
    """Checks a state [B][W][...] whose rows are contiguous; its strides of a sequence and of a
    row, and the bytes of a row."""
    shape, strides, size = x.shape, x.stride(), x.element_size()
    if not x.is_cuda or x.device != dev:
        raise ValueError(f"{name} must be a CUDA tensor on {dev}")
    if len(shape) < 2 or shape[0] != B or shape[1] != W:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected ({B}, {W}, ...)")
    if x.is_contiguous():
        return strides[0] * size, strides[1] * size, math.prod(shape[2:]) * size
    want = 1
    for n, s in zip(reversed(shape[2:]), reversed(strides[2:])):
        if n > 1 and s != want:
            raise ValueError(f"{name} must have contiguous rows")
        want *= n
    return strides[0] * size, strides[1] * size, want * size


@_on_device
def beam_reorder(states, parents, *, out=None, status=None):
    """States [B][W][...] (a tensor or a sequence of up to 16, any types, rows contiguous) in the
    order of parents [B][k] (int32, beam_select's): row i of a sequence is row parents[b][i], and
    for -1 row i itself.  Returns new tensors [B][k][...], or `out`: the same tensors (k = W), to
    reorder them where they are, or memory of their own."""
    single = isinstance(states, torch.Tensor)
    xs = (states,) if single else tuple(states)
    ys = None if out is None else (out,) if single else tuple(out)
    if not xs:
        return [] if out is None else out
    if len(xs) > SD_MAX_STATES or (ys is not None and len(ys) != len(xs)):
        raise ValueError(f"at most {SD_MAX_STATES} states, and as many outputs")
    dev, shape = xs[0].device, parents.shape
    if len(shape) != 2 or xs[0].dim() < 2:
        raise ValueError("parents must be [B][k], states [B][W][...]")
    p = _i32(parents, "parents", shape, dev)
    (B, k), W = shape, xs[0].shape[1]
    if ys is None and k > W:
        raise ValueError("parents has more slots than there are rows: give out")
    a, made = [], []   # the fields of the sd_beam_states, all of 64 bits
    for i, x in enumerate(xs):
        sb, sw, row = _state(x, "states", B, W, dev)
        if ys is None:
            y = torch.empty((B, k, *x.shape[2:]), dtype=x.dtype, device=dev)
            made.append(y)
            a += x.data_ptr(), sb, sw, y.data_ptr(), k * row, row, row
            continue
        y = ys[i]
        if y is not x or k != W:
            if y.dtype != x.dtype or y.shape[2:] != x.shape[2:]:
                raise ValueError("out must have the rows and types of the states")
            to = _state(y, "out", B, k, dev)
        else:
            to = sb, sw, row
        if not (y.is_contiguous() or _lie_apart(row, (B, to[0]), (k, to[1]))):
            raise ValueError("rows of out overlap")
        a += x.data_ptr(), sb, sw, y.data_ptr(), to[0], to[1], row
    if ys is not None:
        if len(ys) > 1 or ys[0] is not xs[0]:
            _apart_or_same(xs, ys)
        if any(_rows_meet(y, parents[None], 2) for y in ys):
            raise ValueError("out overlaps parents")
    st = None if status is None else _i32(status, "status", (1,), dev)
    fields = (ctypes.c_int64 * len(a))(*a)
    rc = _lib().sd_beam_reorder(B, W, k, p, len(xs), ctypes.addressof(fields), st,
                                _stream_of(dev))
    if rc:
        _check(rc, "sd_beam_reorder")
    if out is not None:
        for y in ys:
            _written(y)
        return out
    return made[0] if single else made


def _apart_or_same(xs, ys):
    """Each output is its state itself or shares no memory with any state or other output."""
    for i, y in enumerate(ys):
        for j, x in enumerate(xs):
            if i == j and x.shape == y.shape and _same(x, y):
                continue
            if _rows_meet(x, y, 2):
                raise ValueError("out overlaps a state without being the same tensor")
        if any(_rows_meet(y, z, 2) for z in ys[:i]):
            raise ValueError("outputs overlap")
