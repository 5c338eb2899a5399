"""Python binding of the beam search operators (argument marshalling only)."""
from __future__ import annotations

import ctypes
import math

import torch
from torch.autograd.graph import increment_version

from . import _lib
from .head import _DTYPES, _on


def beam_select(logits: torch.Tensor, score: torch.Tensor, nb: int, *, idx: torch.Tensor | None = None,
                ended: torch.Tensor | None = None, end_id: int = 0):
    """The nb best continuations of each sequence over its beams' columns.

    logits: [B, m, n], bfloat16 or float32, rows evenly spaced and dense
    (a view of the first n columns of wider rows will do); score: [B, m]
    float32 path log probabilities; idx: [B, m, n] int32 ids of candidate
    lists (as Head.draft returns them), None where a column is its own id.
    Probabilities are over the n columns: those of candidate lists are the
    draft distribution's, as branch() gives them, not the vocabulary's.
    ended: [B, m] bool or uint8, beams that only carry on with end_id.
    Returns (score float32, beam int32, token int32), all [B, nb]; see
    lrhead_beam_select in include/lrhead.h.
    """
    for name, v in (("nb", nb), ("end_id", end_id)):
        if not -2 ** 31 <= v < 2 ** 31:   # the C call takes 32 bits, and would get those
            raise ValueError(f"{name} = {v} does not fit int32")
    code = _DTYPES.get(logits.dtype)
    if code is None or not logits.is_cuda or logits.dim() != 3:
        raise ValueError(f"logits must be a bfloat16 or float32 device tensor [B, m, n], not {logits.dtype} "
                         f"{tuple(logits.shape)} on {logits.device}")
    B, m, n = logits.shape
    s0, ld, s2 = logits.stride()
    if m == 1:
        ld = s0
    if B * m <= 1:
        ld = n
    if n < 1 or m < 1 or (n > 1 and s2 != 1) or (B > 1 and m > 1 and s0 != m * ld) or ld < n:
        raise ValueError("logits must be dense rows of an even spacing, with beams and columns")
    dev = logits.device
    if score.dtype != torch.float32 or score.shape != (B, m) or score.device != dev or not score.is_contiguous():
        raise ValueError(f"score must be a contiguous float32 tensor ({B}, {m}) on {dev}")
    if idx is not None and (idx.dtype != torch.int32 or idx.shape != (B, m, n) or idx.device != dev
                            or not idx.is_contiguous()):
        raise ValueError(f"idx must be a contiguous int32 tensor ({B}, {m}, {n}) on {dev}")
    if ended is not None and (ended.dtype not in (torch.uint8, torch.bool) or ended.shape != (B, m)
                              or ended.device != dev or not ended.is_contiguous()):
        raise ValueError(f"ended must be a contiguous bool or uint8 tensor ({B}, {m}) on {dev}")
    lib = _lib.load()
    with _on(dev) as stream:
        ws, nbytes = None, 0
        if n > 64:
            nbytes = lib.lrhead_beam_workspace_bytes(code, B, m, n, nb)
            if nbytes:   # else the call itself says why
                ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        rows = max(nb, 0)
        out = torch.empty((B, rows), dtype=torch.float32, device=dev)
        beam = torch.empty((B, rows), dtype=torch.int32, device=dev)
        token = torch.empty((B, rows), dtype=torch.int32, device=dev)
        rc = lib.lrhead_beam_select(code, logits.data_ptr(), ld, None if idx is None else idx.data_ptr(),
                                    score.data_ptr(), None if ended is None else ended.data_ptr(), end_id, B, m, n, nb,
                                    out.data_ptr(), beam.data_ptr(), token.data_ptr(),
                                    None if ws is None else ws.data_ptr(), nbytes, stream)
        if rc:
            _lib.check(rc, "lrhead_beam_select")
    return out, beam, token


def reorder(states, parent: torch.Tensor, *, length: torch.Tensor | None = None, dim: int = -2, out=None):
    """Beams' states moved behind a selection: out[b, j] = state[b, parent[b, j]].

    states: one tensor [B, m, ...] or a list of them (contiguous, any
    dtype); parent: [B, nb] int32, as beam_select's beam. With length ([B]
    int32) only the first length[b] positions along each state's dimension
    `dim` are moved. What is not moved (positions behind length, slots whose
    parent lies outside [0, m)) keeps what `out` held; without `out` the
    result is new and holds zeros there. See lrhead_reorder.
    """
    single = isinstance(states, torch.Tensor)
    states = [states] if single else list(states)
    if not parent.is_cuda or parent.dtype != torch.int32 or parent.dim() != 2 or not parent.is_contiguous():
        raise ValueError("parent must be a contiguous int32 device tensor [B, nb]")
    dev = parent.device
    B, nb = parent.shape
    given = ()
    if out is None:
        out = [None] * len(states)
    else:
        given = out = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(out) != len(states):
            raise ValueError("out must have one tensor per state")
    if length is not None and (length.device != dev or length.dtype != torch.int32 or length.shape != (B,)
                               or not length.is_contiguous()):
        raise ValueError(f"length must be a contiguous int32 tensor ({B},) on {dev}")
    if not states:
        return []
    m = states[0].shape[1] if states[0].dim() >= 2 else 0
    table = []   # lrhead_state_t, field by field
    with _on(dev) as stream:
        for i, x in enumerate(states):
            shape = x.shape
            if len(shape) < 2 or shape[0] != B or shape[1] != m or x.device != dev or not x.is_contiguous():
                raise ValueError(f"state {i} must be a contiguous tensor [{B}, {m}, ...] on {dev}")
            o = out[i]
            if o is None:
                o = out[i] = torch.zeros((B, nb, *shape[2:]), dtype=x.dtype, device=dev)
            elif (o.dtype != x.dtype or o.shape[:2] != (B, nb) or o.shape[2:] != shape[2:] or o.device != dev
                  or not o.is_contiguous()):
                raise ValueError(f"out {i} must be a contiguous {x.dtype} tensor {(B, nb, *shape[2:])} on {dev}")
            if length is None:
                table += (x.data_ptr(), o.data_ptr(), 1, 1, math.prod(shape[2:]) * x.element_size())
            else:
                d = dim + len(shape) if dim < 0 else dim
                if not 2 <= d < len(shape):
                    raise ValueError(f"state {i} has no dimension {dim} behind its beams")
                table += (x.data_ptr(), o.data_ptr(), math.prod(shape[2:d]), shape[d],
                          math.prod(shape[d + 1:]) * x.element_size())
        if nb and m:
            rc = _lib.load().lrhead_reorder((ctypes.c_int64 * len(table))(*table), len(states), parent.data_ptr(),
                                            None if length is None else length.data_ptr(), B, m, nb, stream)
            if rc:
                _lib.check(rc, "lrhead_reorder")
            if given:
                increment_version(given)   # so that autograd knows of the change
    return out[0] if single else out
