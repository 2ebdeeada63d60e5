"""ctypes marshalling for beam search: the choice of the next hypotheses, and the reordering
of the beams' states after it (see include/vce.h for what each computes).  The conventions
are those of ``_head``.
"""
from __future__ import annotations

from array import array
from collections import namedtuple
from functools import lru_cache

import torch

from . import _binding as b
from ._head import (SAMPLE_MAX_VOCAB, MXTensor, _check_head, _float_code, _head_logits, _launch, _status, _under,
                    _vector)

BEAM_MAX_BEAMS, BEAM_MAX_COUNT = 32, 64

CEBeam = namedtuple("CEBeam", "token parent score ended length dev_status")


@lru_cache(maxsize=1024)
def ce_beam_workspace_size(batch: int, beams: int, count: int) -> int:
    return int(b.library().ce_beam_workspace_size(batch, beams, count))


def _beam_args(score, ended, length, end, length_penalty, count, keep_places, vocab, index):
    """Checks what ce_beam takes beside the logits; returns (batch, beams, count, end)."""
    if score.dim() < 1 or score.dtype is not torch.float32 or score.get_device() != index or not score.is_contiguous():
        raise ValueError("score must be a contiguous float32 tensor [..., beams] on the logits' device")
    beams = score.shape[-1]
    if not 1 <= beams <= BEAM_MAX_BEAMS:
        raise ValueError(f"score must have 1 to {BEAM_MAX_BEAMS} beams, got {beams}")
    if not 1 <= vocab <= SAMPLE_MAX_VOCAB:
        raise ValueError(f"the vocabulary must have 1 to {SAMPLE_MAX_VOCAB} tokens, got {vocab}")
    rows = score.numel()
    count = beams if count is None else count
    end = -1 if end is None else end
    if count != int(count) or not 1 <= count <= BEAM_MAX_COUNT:
        raise ValueError(f"count must be a whole number from 1 to {BEAM_MAX_COUNT}, got {count}")
    if keep_places and count != beams:
        raise ValueError(f"keep_places needs as many hypotheses as beams ({beams}), got {count}")
    if end != int(end) or not -1 <= end < vocab:
        raise ValueError(f"end must be a token, or -1, got {end}")
    if ended is not None:
        _vector(ended, "ended", rows, torch.bool, index)
        if end < 0:
            raise ValueError("ended needs end, the token that an ended hypothesis goes on with")
    if length is not None:
        _vector(length, "length", rows, torch.int32, index)
    if not -16 <= length_penalty <= 16:
        raise ValueError(f"length_penalty must be between -16 and 16, got {length_penalty}")
    if length_penalty and length is None:
        raise ValueError("length_penalty needs length")
    return rows // beams, beams, int(count), int(end)


def _outputs(dev, index, args, score, ended, length, out):
    """The outputs, checked where they are given: token, parent, score, ended, length."""
    _, beams, count, end = args
    shape, n = (*score.shape[:-1], count), score.numel() // beams * count
    token, parent, out_score, out_ended, out_length = out

    def written(t, name, dtype):
        return torch.empty(shape, dtype=dtype, device=dev) if t is None else _vector(t, name, n, dtype, index)

    token, parent = written(token, "token", torch.int64), written(parent, "parent", torch.int64)
    out_score = written(out_score, "out_score", torch.float32)
    if ended is not None or end >= 0:
        out_ended = written(out_ended, "out_ended", torch.bool)
    elif out_ended is not None:
        raise ValueError("out_ended is written only when ended or end is given")
    if length is not None:
        out_length = written(out_length, "out_length", torch.int32)
    elif out_length is not None:
        raise ValueError("out_length is written only when length is given")
    return token, parent, out_score, out_ended, out_length


def _choose(logits, code, vocab, stride, args, score, ended, length, length_penalty, keep_places, out, workspace, status):
    """The library's call, all arguments checked."""
    dev = logits.device
    batch, beams, count, end = args
    token, parent, out_score, out_ended, out_length = out
    lib, ptr = b.library(), b._ptr
    if workspace is None:
        workspace = torch.empty(ce_beam_workspace_size(batch, beams, count) or 1, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != logits.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the logits' device")
    _launch("ce_beam", dev, lib.ce_beam, logits.data_ptr(), code, batch, beams, vocab, stride, score.data_ptr(),
            ptr(ended), ptr(length), end, length_penalty, count, int(bool(keep_places)), token.data_ptr(),
            parent.data_ptr(), out_score.data_ptr(), ptr(out_ended), ptr(out_length), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), status)


def ce_beam(logits, score, *, ended=None, length=None, end=-1, length_penalty=0.0, count=None, keep_places=False,
            token=None, parent=None, out_score=None, out_ended=None, out_length=None, workspace=None, dev_status=None,
            stream=None):
    """The next ``count`` (default: as many as beams) hypotheses of every request from ``logits``
    [..., V] (bfloat16 or float32), a row per beam, and ``score`` [..., beams] (float32).

    A beam offers every token v with its score plus log softmax(logits)_v, and its ``length``
    (int32, like score) plus one; one that has ``ended`` (bool, like score) offers itself.  The
    best by score / length^length_penalty are taken, lowest (beam, token) first among equals.
    ``end`` is the token with which a hypothesis ends.  A score of -inf marks a beam that
    offers nothing.  With ``keep_places`` a beam's first child stays at its parent's place,
    so that beam_reorder moves little.

    Returns (token int64, parent int64, score, ended, length, dev_status), shaped like score with
    ``count`` in the last place; parent is an index among the request's beams.  ended is None
    where neither ``ended`` nor ``end`` is given, length where ``length`` is not.  The state of
    a search can be updated in place where count is beams: out_score=score, out_ended=ended, out_length=length.
    Places for which nothing is offered get token -1 and score -inf.  A beam whose logits give
    no distribution offers nothing and sets a bit of ``dev_status`` (int32 [1]) where passed."""
    if stream is not None:
        return _under(stream, ce_beam, logits, score, ended=ended, length=length, end=end, length_penalty=length_penalty,
                      count=count, keep_places=keep_places, token=token, parent=parent, out_score=out_score,
                      out_ended=out_ended, out_length=out_length, workspace=workspace, dev_status=dev_status)
    code = _float_code(logits.dtype, "logits")
    n, vocab, stride = b._rows_view(logits)
    index = logits.get_device()
    args = _beam_args(score, ended, length, end, length_penalty, count, keep_places, vocab, index)
    if n != score.numel():
        raise ValueError(f"logits have {n} rows, score {score.numel()} beams")
    out = _outputs(logits.device, index, args, score, ended, length, (token, parent, out_score, out_ended, out_length))
    _choose(logits, code, vocab, stride, args, score, ended, length, length_penalty, keep_places, out, workspace,
            _status(dev_status, index))
    return CEBeam(*out, dev_status)


def linear_beam(embeddings, classifier: MXTensor, score, *, ended=None, length=None, end=-1, length_penalty=0.0,
                count=None, keep_places=False, norm_weight=None, norm_eps=1e-6, residual=None, adapters=None,
                adapter_index=None, out_score=None, out_ended=None, out_length=None, dev_status=None, stream=None):
    """The next hypotheses after ``embeddings`` [..., H], a row per beam: linear_sample's norm, product
    and adapters, and ce_beam of the logits.  Returns ce_beam's results, with a zeroed ``dev_status``
    of its own where none is passed: mx_linear's bits are in it too."""
    if stream is not None:
        return _under(stream, linear_beam, embeddings, classifier, score, ended=ended, length=length, end=end,
                      length_penalty=length_penalty, count=count, keep_places=keep_places, norm_weight=norm_weight,
                      norm_eps=norm_eps, residual=residual, adapters=adapters, adapter_index=adapter_index,
                      out_score=out_score, out_ended=out_ended, out_length=out_length, dev_status=dev_status)
    n, v, index = _check_head(embeddings, classifier, norm_weight, residual, adapters, adapter_index, dev_status)
    args = _beam_args(score, ended, length, end, length_penalty, count, keep_places, v, index)
    if n != score.numel():
        raise ValueError(f"embeddings have {n} rows, score {score.numel()} beams")
    out = _outputs(embeddings.device, index, args, score, ended, length, (None, None, out_score, out_ended, out_length))
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=embeddings.device)
    logits = _head_logits(embeddings, classifier, n, v, norm_weight, norm_eps, residual, adapters, adapter_index,
                          dev_status)
    _choose(logits, b.F32, v, logits.stride(0), args, score, ended, length, length_penalty, keep_places, out, None,
            dev_status.data_ptr())
    return CEBeam(*out, dev_status)


# ---------------------------------------------------------------------------
# the beams' states
# ---------------------------------------------------------------------------

def _merge(dims):
    """(size, stride) of ``dims`` [(size, stride), ...] as one dimension, None if they are none."""
    dims = [d for d in dims if d[0] != 1]
    if not dims:
        return 1, 0
    for (_, outer), (size, inner) in zip(dims, dims[1:]):
        if outer != size * inner:
            return None
    size = 1
    for d in dims:
        size *= d[0]
    return size, dims[-1][1]


@lru_cache(maxsize=1024)
def _layout(shape, strides, itemsize, position_dim):
    """(row stride, parts, part stride, positions, position bytes) of a state, in bytes, and
    whether its elements all lie at places of their own; a text where the library cannot take it."""
    dims = list(zip(shape[1:], strides[1:]))
    if 0 in shape[1:]:
        return (0, 0, 0, 0, 0), True
    if position_dim is None:  # the innermost contiguous run
        at, expect = len(dims), 1
        while at > 0 and (dims[at - 1][0] == 1 or dims[at - 1][1] == expect):
            expect *= dims[at - 1][0]
            at -= 1
        positions, each = 1, expect
    else:
        if not 1 <= position_dim < len(shape):
            return f"position_dim must be one of a row's dimensions, got {position_dim} for {len(shape)} dimensions"
        at, each = position_dim - 1, 1
        for size, stride in reversed(dims[at + 1:]):
            if size != 1 and stride != each:
                return "what belongs to a position must be contiguous"
            each *= size
        positions, stride = dims[at]
        if positions != 1 and stride != each:
            return "the positions of a state must follow one another"
    outer = _merge(dims[:at])
    if outer is None:
        return "the dimensions around the positions must have one stride"
    (parts, part), run, rows, row = outer, positions * each, shape[0], strides[0] if shape[0] > 1 else 0
    levels = sorted([(s, n) for s, n in ((part, parts), (row, rows)) if n > 1])
    extent, apart = run, True
    for stride, n in levels:
        apart = apart and stride >= extent
        extent += stride * (n - 1)
    return (row * itemsize, parts, part * itemsize, positions, each * itemsize), apart


def _state_layout(t, dim, rows, index, name):
    if t.dim() < 1 or t.shape[0] != rows or t.get_device() != index:
        raise ValueError(f"{name} must have a row for each of the {rows} beams, on parent's device, got "
                         f"{tuple(t.shape)} on {t.device}")
    layout = _layout(t.shape, t.stride(), t.element_size(), dim)
    if isinstance(layout, str):
        raise ValueError(f"{name}: {layout}")
    return layout


def beam_reorder(states, parent, *, lengths=None, position_dim=None, out=None, dev_status=None, stream=None):
    """Gives every beam its parent's states: row (request, k) of each state becomes the row
    (request, parent[request, k]).  ``states`` is a tensor or a list of tensors of any type with a
    row for each beam in their first dimension, request by request; ``parent`` int64 [..., beams].

    In place (beams that keep their place are not touched), or into ``out``, tensors like the
    states that share no memory with them.  What is written shares none with another state, parent or
    lengths either.  With ``lengths`` (int32, one per request) only the first so many
    positions move, along ``position_dim`` (a number, or one for each state): for keys
    [rows, heads, T, D] it is 2, for [rows, T, heads, D] it is 1.  Positions must follow one another in
    memory, and the dimensions before them have one stride.  An entry of parent that names no beam
    counts as the beam itself and sets a bit of ``dev_status``.  Returns what was written."""
    if stream is not None:
        return _under(stream, lambda p, **kw: beam_reorder(states, p, **kw), parent, lengths=lengths,
                      position_dim=position_dim, out=out, dev_status=dev_status)
    single = isinstance(states, torch.Tensor)
    srcs = [states] if single else list(states)
    dsts = srcs if out is None else [out] if single else list(out)
    dims = [position_dim] * len(srcs) if position_dim is None or isinstance(position_dim, int) else list(position_dim)
    if len(dsts) != len(srcs) or len(dims) != len(srcs):
        raise ValueError(f"{len(srcs)} states, {len(dsts)} in out, {len(dims)} in position_dim")
    dev, index = parent.device, parent.get_device()
    if parent.dim() < 1 or parent.dtype is not torch.int64 or not parent.is_contiguous():
        raise ValueError("parent must be a contiguous int64 tensor [..., beams]")
    rows, beams = parent.numel(), parent.shape[-1]
    if not 1 <= beams <= BEAM_MAX_BEAMS:
        raise ValueError(f"parent must have 1 to {BEAM_MAX_BEAMS} beams, got {beams}")
    batch = rows // beams
    if lengths is not None:
        _vector(lengths, "lengths", batch, torch.int32, index)
    written, read = set(), set()
    packed, last = [], None  # (a cache's tensors are mostly alike: what was found out of one holds for the next)
    for src, dst, dim in zip(srcs, dsts, dims):
        if lengths is not None and dim is None:
            raise ValueError("lengths need the position_dim of every state")
        kind = (src.shape, src.stride(), src.dtype, dim, src.get_device())
        if kind != last:
            (row, parts, part, positions, each), apart = _state_layout(src, dim, rows, index, "a state")
            last = kind
        at = src.data_ptr()
        if dst is src:
            if not apart or at in written:
                raise ValueError("a state that is written has elements that share memory, or is there twice")
            if positions:
                written.add(at)
            packed += (at, at, row, row, parts, part, part, positions, each)
            continue
        if dst.shape != src.shape or dst.dtype is not src.dtype:
            raise ValueError(f"out must match the states: {dst.dtype}, {tuple(dst.shape)} for {src.dtype}, {tuple(src.shape)}")
        (to_row, to_parts, to_part, *run), to_apart = _state_layout(dst, dim, rows, index, "out")
        to = dst.data_ptr()
        if parts != to_parts or run != [positions, each]:
            raise ValueError("a state and its out must divide into the same contiguous runs")
        if to == at and (row, part) != (to_row, to_part):
            raise ValueError("out shares memory with its state")
        if not to_apart or to in written:
            raise ValueError("an out has elements that share memory, or is there twice")
        if positions:
            written.add(to)
            if at != to:
                read.add(at)
        packed += (at, to, row, to_row, parts, part, to_part, positions, each)
    if not written.isdisjoint(read):
        raise ValueError("out shares memory with the states")
    states_of = array("q", packed)  # vce_state: nine 64-bit words
    _launch("beam_reorder", dev, b.library().beam_reorder, states_of.buffer_info()[0], len(srcs), parent.data_ptr(),
            batch, beams, b._ptr(lengths), _status(dev_status, index))
    return dsts[0] if single else dsts
