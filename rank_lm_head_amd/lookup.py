"""Python binding of the embedding lookup and its gradient (argument marshalling only)."""
from __future__ import annotations

import math

import torch
from torch.autograd.forward_ad import unpack_dual
from torch.autograd.graph import increment_version

from . import _lib
from .head import _DTYPES, _on


def _scale(scale) -> float:
    scale = float(scale)
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, not {scale}")
    return scale


def embed(W: torch.Tensor, token: torch.Tensor, *, scale: float = 1.0) -> torch.Tensor:
    """scale * W[token]: [*token.shape, d] in W's dtype; zeros for a token
    outside [0, V), as sample, verify and beam_select mark empty slots.

    W: [V, d], bfloat16 or float32, contiguous; token: int32, of any shape,
    contiguous. Not differentiable (see embedding()). See lrhead_embed in
    include/lrhead.h.
    """
    code = _DTYPES.get(W.dtype)
    if code is None or not W.is_cuda or W.dim() != 2 or not W.is_contiguous():
        raise ValueError(f"W must be a contiguous bfloat16 or float32 device matrix, not {W.dtype} {tuple(W.shape)} "
                         f"on {W.device}")
    dev = W.device
    if token.dtype != torch.int32 or token.device != dev or not token.is_contiguous():
        raise ValueError(f"token must be a contiguous int32 tensor on {dev}")
    V, d = W.shape
    lib = _lib.load()
    with _on(dev) as stream:
        out = torch.empty((*token.shape, d), dtype=W.dtype, device=dev)
        rc = lib.lrhead_embed(code, W.data_ptr(), V, d, token.data_ptr(), token.numel(), _scale(scale), out.data_ptr(),
                              stream)
        if rc:
            _lib.check(rc, "lrhead_embed")
    return out


def embed_grad(dY: torch.Tensor, token: torch.Tensor, V: int, *, scale: float = 1.0,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of W in embed(W, token, scale=scale), [V, d], from dY
    ([*token.shape, d], contiguous): new, or added to `out`, of which only the
    rows of tokens that occur are touched. Sums are float32 and rounded once,
    in an order that does not vary. See lrhead_embed_grad in
    include/lrhead.h."""
    code = _DTYPES.get(dY.dtype)
    if code is None or not dY.is_cuda or dY.dim() < 1 or not dY.is_contiguous():
        raise ValueError(f"dY must be a contiguous bfloat16 or float32 device tensor, not {dY.dtype} on {dY.device}")
    dev, d = dY.device, dY.shape[-1]
    if token.dtype != torch.int32 or token.shape != dY.shape[:-1] or token.device != dev or not token.is_contiguous():
        raise ValueError(f"token must be a contiguous int32 tensor {tuple(dY.shape[:-1])} on {dev}")
    if not 1 <= V < 2 ** 31:
        raise ValueError(f"V = {V} outside [1, 2^31)")
    if out is not None and (out.dtype != dY.dtype or out.shape != (V, d) or out.device != dev
                            or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous {dY.dtype} tensor ({V}, {d}) on {dev}")
    N = token.numel()
    lib = _lib.load()
    with _on(dev) as stream:
        nbytes = lib.lrhead_embed_grad_workspace_bytes(code, V, d, N)
        # without sizes that can be, the call itself says why
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        dW = torch.empty((V, d) if nbytes else (1, 1), dtype=dY.dtype, device=dev) if out is None else out
        rc = lib.lrhead_embed_grad(code, dY.data_ptr(), token.data_ptr(), N, V, d, _scale(scale), out is not None,
                                   dW.data_ptr(), None if ws is None else ws.data_ptr(), nbytes, stream)
        if rc:
            _lib.check(rc, "lrhead_embed_grad")
    if out is not None:
        increment_version(out)   # so that autograd knows of the change
    return dW


def _no_capture(device) -> None:
    # Under graph capture autograd's own accumulation nodes may belong to
    # another stream; the process would end, so the call is refused.
    with _on(device):
        capturing = torch.cuda.is_current_stream_capturing()
    if capturing:
        raise RuntimeError("embedding cannot be captured with gradients; capture embed and embed_grad")


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, W, token, scale):
        if W.is_cuda:   # else embed() says so
            _no_capture(W.device)
        ctx.save_for_backward(token)
        ctx.V, ctx.scale = W.shape[0], scale
        return embed(W, token, scale=scale)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        token, = ctx.saved_tensors
        _no_capture(g.device)
        return embed_grad(g.contiguous(), token, ctx.V, scale=ctx.scale), None, None


def embedding(W: torch.Tensor, token: torch.Tensor, *, scale: float = 1.0) -> torch.Tensor:
    """embed(), differentiable in W (backwards only: a W with a forward-mode
    tangent is refused). Not for graph capture with gradients: capture embed
    and embed_grad."""
    # a tangent does not show in requires_grad, and no_grad does not end it
    if unpack_dual(W).tangent is not None:
        raise NotImplementedError("embedding has no forward-mode derivative")
    if not (torch.is_grad_enabled() and W.requires_grad):
        return embed(W, token, scale=scale)
    return _Embedding.apply(W, token, _scale(scale))
