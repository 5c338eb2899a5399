"""Python binding of sampling and verification (argument marshalling only)."""
from __future__ import annotations

import torch

from . import _lib
from .head import _DTYPES, _on


def _settings(temperature, top_k, top_p, min_p, rows: int, dev) -> _lib.Sampling:
    """lrhead_sampling_t of settings that are numbers or [rows] tensors."""
    ptr, one = [None] * 4, [1.0, 0, 1.0, 0.0]
    for i, (name, v) in enumerate((("temperature", temperature), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p))):
        if isinstance(v, torch.Tensor):
            dtype = torch.int32 if i == 1 else torch.float32
            if v.dtype != dtype or v.shape != (rows,) or v.device != dev or not v.is_contiguous():
                raise ValueError(f"{name} must be a number or a contiguous {dtype} tensor ({rows},) on {dev}")
            ptr[i] = v.data_ptr()
        elif i == 1 and not -2 ** 31 <= v < 2 ** 31:   # the C call takes 32 bits, and would get those
            raise ValueError(f"top_k = {v} does not fit int32")
        else:
            one[i] = v
    return _lib.Sampling(*ptr, *one)


def _spacing(logits: torch.Tensor) -> int:
    """Elements from row to row of [..., n]: dense rows of an even spacing."""
    n = logits.shape[-1]
    if n < 1 or (n > 1 and logits.stride(-1) != 1):
        raise ValueError("logits must be dense rows, with columns")
    if logits.dim() == 2:
        ld = logits.stride(0) if logits.shape[0] > 1 else n
    else:
        B, m, _ = logits.shape
        ld = logits.stride(1) if m > 1 else logits.stride(0) if B > 1 else n
        if B > 1 and m > 1 and logits.stride(0) != m * ld:
            raise ValueError("logits must be rows of an even spacing")
    if ld < n:
        raise ValueError("logits must be rows of an even spacing that do not overlap")
    return ld


def sample(logits: torch.Tensor, u: torch.Tensor, *, idx: torch.Tensor | None = None, temperature=1.0, top_k=0,
           top_p=1.0, min_p=0.0, want_probs: bool = False):
    """A token of each row of logits, drawn with the given random numbers.

    logits: [B, n], bfloat16 or float32, rows evenly spaced and dense; u:
    [B] float32 in [0, 1); idx: [B, n] int32 ids of candidate lists (as
    Head.draft returns them), None where a column is its own id.
    temperature (0: greedy), top_k (0: all), top_p and min_p are numbers or
    [B] tensors (float32, top_k int32). Returns (token int32 [B], prob float32
    [B], probs float32 [B, n] or None): the token (-1 for a row without
    candidates), its probability among what the settings leave in, and with
    want_probs, for rows of at most 64 columns, that of every column. See
    lrhead_sample in include/lrhead.h.
    """
    code = _DTYPES.get(logits.dtype)
    if code is None or not logits.is_cuda or logits.dim() != 2:
        raise ValueError(f"logits must be a bfloat16 or float32 device tensor [B, n], not {logits.dtype} "
                         f"{tuple(logits.shape)} on {logits.device}")
    B, n = logits.shape
    ld = _spacing(logits)
    dev = logits.device
    if u.dtype != torch.float32 or u.shape != (B,) or u.device != dev or not u.is_contiguous():
        raise ValueError(f"u must be a contiguous float32 tensor ({B},) on {dev}")
    if idx is not None and (idx.dtype != torch.int32 or idx.shape != (B, n) or idx.device != dev
                            or not idx.is_contiguous()):
        raise ValueError(f"idx must be a contiguous int32 tensor ({B}, {n}) on {dev}")
    if want_probs and n > _lib.K_MAX:
        raise ValueError(f"probabilities of all columns are for rows of at most {_lib.K_MAX}, not {n}")
    how = _settings(temperature, top_k, top_p, min_p, B, dev)
    lib = _lib.load()
    with _on(dev) as stream:
        ws, nbytes = None, 0
        if n > _lib.K_MAX:
            nbytes = lib.lrhead_sample_workspace_bytes(code, B, n)
            if nbytes:   # else the call itself says why
                ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        token = torch.empty(B, dtype=torch.int32, device=dev)
        prob = torch.empty(B, dtype=torch.float32, device=dev)
        probs = torch.empty((B, n), dtype=torch.float32, device=dev) if want_probs else None
        rc = lib.lrhead_sample(code, logits.data_ptr(), ld, None if idx is None else idx.data_ptr(), u.data_ptr(), how,
                               B, n, token.data_ptr(), prob.data_ptr(), None if probs is None else probs.data_ptr(),
                               None if ws is None else ws.data_ptr(), nbytes, stream)
        if rc:
            _lib.check(rc, "lrhead_sample")
    return token, prob, probs


def verify(logits: torch.Tensor, token: torch.Tensor, u: torch.Tensor, *, idx: torch.Tensor | None = None,
           probs: torch.Tensor | None = None, length: torch.Tensor | None = None, temperature=1.0, top_k=0, top_p=1.0,
           min_p=0.0):
    """Drafted tokens accepted or replaced so that what comes out is
    distributed as the target's own samples under the settings.

    logits: the target's, [B, s+1, n], bfloat16 or float32, rows evenly spaced
    and dense; token: [B, s] int32 drafted tokens; u: [B, s+1] float32 in
    [0, 1), the last of a sequence for its draw; idx, probs: [B, s, k] the
    candidate lists that the tokens were drawn from (int32 ids and float32
    probabilities, as sample() returns them), None for tokens of probability
    1; length: [B] int32 drafted tokens that there are (None: s). The
    settings are sample()'s, numbers or [B] tensors. Returns (token int32
    [B, s+1], -1 behind the last; count int32 [B]). See lrhead_verify in
    include/lrhead.h.
    """
    code = _DTYPES.get(logits.dtype)
    if code is None or not logits.is_cuda or logits.dim() != 3:
        raise ValueError(f"logits must be a bfloat16 or float32 device tensor [B, s + 1, n], not {logits.dtype} "
                         f"{tuple(logits.shape)} on {logits.device}")
    B, m, n = logits.shape
    s = m - 1
    if s < 0:
        raise ValueError("logits must have a row of each sequence at least")
    ld = _spacing(logits)
    dev = logits.device
    k = 1
    if (idx is None) != (probs is None):
        raise ValueError("idx and probs go together")
    if idx is not None:
        if idx.dim() != 3:
            raise ValueError(f"idx must be ({B}, {s}, k), not {tuple(idx.shape)}")
        k = idx.shape[2]
        if k < 1:   # an empty tensor has no address, and the C call would take the lists as left out
            raise ValueError("idx must have a column at least")
    for name, t, dtype, shape in (("token", token, torch.int32, (B, s)), ("u", u, torch.float32, (B, m)),
                                  ("idx", idx, torch.int32, (B, s, k)), ("probs", probs, torch.float32, (B, s, k)),
                                  ("length", length, torch.int32, (B,))):
        if t is not None and (t.dtype != dtype or t.shape != shape or t.device != dev or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {shape} on {dev}")
    how = _settings(temperature, top_k, top_p, min_p, B, dev)
    lib = _lib.load()
    with _on(dev) as stream:
        nbytes = lib.lrhead_verify_workspace_bytes(code, B, s, n)
        # without sizes that can be, the call itself says why
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        out = torch.empty((B, m), dtype=torch.int32, device=dev)
        count = torch.empty(B, dtype=torch.int32, device=dev)
        rc = lib.lrhead_verify(code, logits.data_ptr(), ld, token.data_ptr(), None if idx is None else idx.data_ptr(),
                               None if probs is None else probs.data_ptr(), k,
                               None if length is None else length.data_ptr(), u.data_ptr(), how, B, s, n,
                               out.data_ptr(), count.data_ptr(), None if ws is None else ws.data_ptr(), nbytes, stream)
        if rc:
            _lib.check(rc, "lrhead_verify")
    return out, count
