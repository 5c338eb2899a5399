"""Python binding of the beam search operators (argument marshalling only)."""
from __future__ import annotations

import math

import torch

from . import _lib
from .head import _DTYPES, _need, _on, _ptr


def beam_select(logits: torch.Tensor, score: torch.Tensor, nb: int, *, idx: torch.Tensor | None = None,
                ended: torch.Tensor | None = None, end_id: int = 0):
    """The nb best continuations of each sequence over its beams' columns.

    logits: [B, m, n], bfloat16 or float32, rows evenly spaced and dense
    (a view of the first n columns of wider rows will do); score: [B, m]
    float32 path log probabilities; idx: [B, m, n] int32 ids of candidate
    lists (as Head.draft returns them), None where a column is its own id;
    ended: [B, m] bool or uint8, beams that only carry on with end_id.
    Returns (score float32, beam int32, token int32), all [B, nb]; see
    lrhead_beam_select in include/lrhead.h.
    """
    _need(logits.dtype in _DTYPES, f"unsupported dtype {logits.dtype}")
    _need(logits.is_cuda and logits.dim() == 3, "logits must be a device tensor [B, m, n]")
    B, m, n = logits.shape
    _need(n >= 1 and m >= 1, "logits must have beams and columns")
    ld = logits.stride(1) if m > 1 else logits.stride(0) if B > 1 else n
    _need((n == 1 or logits.stride(2) == 1) and (B <= 1 or m == 1 or logits.stride(0) == m * ld) and (B * m <= 1 or ld >= n),
          "logits must be dense rows of an even spacing")
    dev = logits.device
    want = [("score", score, (B, m), (torch.float32,))]
    if idx is not None:
        want.append(("idx", idx, (B, m, n), (torch.int32,)))
    if ended is not None:
        want.append(("ended", ended, (B, m), (torch.uint8, torch.bool)))
    for name, t, shape, dtypes in want:
        _need(t.dtype in dtypes and tuple(t.shape) == shape and t.device == dev and t.is_contiguous(),
              f"{name} must be a contiguous {dtypes[0]} tensor of shape {shape} on {dev}")
    lib = _lib.load()
    code = _DTYPES[logits.dtype]
    with _on(dev) as stream:
        nbytes = lib.lrhead_beam_workspace_bytes(code, B, m, n, nb)
        if nbytes == 0:   # the call itself says why
            _lib.check(lib.lrhead_beam_select(code, None, n, None, None, None, 0, B, m, n, nb, None, None, None, None,
                                              0, None), "lrhead_beam_workspace_bytes")
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        out = torch.empty((B, nb), dtype=torch.float32, device=dev)
        beam = torch.empty((B, nb), dtype=torch.int32, device=dev)
        token = torch.empty((B, nb), dtype=torch.int32, device=dev)
        _lib.check(lib.lrhead_beam_select(code, _ptr(logits), max(ld, n), _ptr(idx), _ptr(score), _ptr(ended), end_id,
                                          B, m, n, nb, _ptr(out), _ptr(beam), _ptr(token), _ptr(ws), nbytes, stream),
                   "lrhead_beam_select")
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
    _need(parent.is_cuda and parent.dtype == torch.int32 and parent.dim() == 2 and parent.is_contiguous(),
          "parent must be a contiguous int32 device tensor [B, nb]")
    dev = parent.device
    B, nb = parent.shape
    _need(len(states) <= _lib.STATES_MAX, f"at most {_lib.STATES_MAX} states")
    if out is None:
        out = [None] * len(states)
    else:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        _need(len(out) == len(states), "out must have one tensor per state")
    if length is not None:
        _need(length.device == dev and length.dtype == torch.int32 and tuple(length.shape) == (B,)
              and length.is_contiguous(), f"length must be a contiguous int32 tensor of shape ({B},) on {dev}")
    if not states:
        return []
    m = states[0].shape[1] if states[0].dim() >= 2 else 0
    arr = (_lib.State * len(states))()
    with _on(dev) as stream:
        for i, x in enumerate(states):
            _need(x.device == dev and x.dim() >= 2 and x.shape[0] == B and x.shape[1] == m and x.is_contiguous(),
                  f"state {i} must be a contiguous tensor [{B}, {m}, ...] on {dev}")
            shape = (B, nb, *x.shape[2:])
            if out[i] is None:
                out[i] = torch.zeros(shape, dtype=x.dtype, device=dev)
            o = out[i]
            _need(o.device == dev and o.dtype == x.dtype and tuple(o.shape) == shape and o.is_contiguous(),
                  f"out {i} must be a contiguous {x.dtype} tensor {shape} on {dev}")
            s = arr[i]
            s.src, s.dst = x.data_ptr(), o.data_ptr()
            if length is None:
                s.segs, s.positions, s.position_bytes = 1, 1, math.prod(x.shape[2:]) * x.element_size()
            else:
                d = dim + x.dim() if dim < 0 else dim
                _need(2 <= d < x.dim(), f"state {i} has no dimension {dim} behind its beams")
                s.segs, s.positions = math.prod(x.shape[2:d]), x.shape[d]
                s.position_bytes = math.prod(x.shape[d + 1:]) * x.element_size()
        if nb and m:
            _lib.check(_lib.load().lrhead_reorder(arr, len(states), _ptr(parent), _ptr(length), B, m, nb, stream),
                       "lrhead_reorder")
    return out[0] if single else out
