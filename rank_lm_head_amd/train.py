"""Python binding of the head's distillation (argument marshalling only).

distill / distill_grad are the two calls of include/lrhead.h; distill_loss
joins them for torch's autograd.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .head import _DTYPES, _need, _on, _ptr


def _check(Z: torch.Tensor, P: torch.Tensor, idx: torch.Tensor, logits: torch.Tensor):
    _need(Z.dtype in _DTYPES and P.dtype == Z.dtype, "Z and P must share a supported dtype (bfloat16 or float32)")
    _need(Z.is_cuda, "Z must be a device tensor")
    _need(Z.dim() == 2 and P.dim() == 2 and P.shape[1] == Z.shape[1], "Z must be (N, r) and P (V, r)")
    N = Z.shape[0]
    _need(idx.dtype == torch.int32 and logits.dtype == torch.float32, "idx must be int32 and logits float32")
    _need(idx.dim() == 2 and idx.shape[0] == N and logits.shape == idx.shape, f"idx and logits must be ({N}, k)")
    for name, t in (("Z", Z), ("P", P), ("idx", idx), ("logits", logits)):
        _need(t.device == Z.device and t.is_contiguous(), f"{name} must be contiguous on {Z.device}")
    return N, int(P.shape[0]), int(Z.shape[1]), int(idx.shape[1])


def _workspace(lib, code, V, r, N, k, device):
    n = lib.lrhead_distill_workspace_bytes(code, V, r, N, k)
    if n == 0:   # the call itself says why
        _lib.check(lib.lrhead_distill(code, V, r, None, None, N, None, None, k, 1.0, None, None, None, None, 0, None),
                   "lrhead_distill_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def distill(Z: torch.Tensor, P: torch.Tensor, idx: torch.Tensor, logits: torch.Tensor, *, temperature: float = 1.0,
            want_grad: bool = True):
    """The loss of the rows Z ([N, r]) under the head P ([V, r]) against a
    teacher's top logits (idx int32 and logits float32, [N, k], as
    Head.full_topk returns them; an id outside [0, V) marks an empty place):
    (loss [N], lse [N], dloss/dZ [N, r] or None), float32. See lrhead_distill
    in include/lrhead.h."""
    N, V, r, k = _check(Z, P, idx, logits)
    lib = _lib.load()
    code, dev = _DTYPES[Z.dtype], Z.device
    with _on(dev) as stream:
        ws = _workspace(lib, code, V, r, N, k, dev)
        loss = torch.empty(N, dtype=torch.float32, device=dev)
        lse = torch.empty(N, dtype=torch.float32, device=dev)
        grad = torch.empty((N, r), dtype=torch.float32, device=dev) if want_grad else None
        _lib.check(lib.lrhead_distill(code, V, r, _ptr(P), _ptr(Z), N, _ptr(idx), _ptr(logits), k, temperature,
                                      _ptr(loss), _ptr(lse), _ptr(grad), _ptr(ws), ws.numel(), stream),
                   "lrhead_distill")
    return loss, lse, grad


def distill_grad(Z: torch.Tensor, P: torch.Tensor, idx: torch.Tensor, logits: torch.Tensor, lse: torch.Tensor,
                 grad: torch.Tensor | None, weight: torch.Tensor | None = None, *, temperature: float = 1.0,
                 want_dZ: bool = True, want_dP: bool = True):
    """The gradients of sum(weight * loss): (dZ [N, r] or None, dP [V, r] or
    None) in Z's dtype, from lse and grad of distill() on the same inputs
    (grad may be None without dZ). weight: [N] float32, None for ones. See
    lrhead_distill_grad in include/lrhead.h."""
    N, V, r, k = _check(Z, P, idx, logits)
    dev = Z.device
    want = [("lse", lse, (N,))]
    if want_dZ:
        _need(grad is not None, "dZ needs the grad of distill()")
        want.append(("grad", grad, (N, r)))
    if weight is not None:
        want.append(("weight", weight, (N,)))
    for name, t, shape in want:
        _need(t.dtype == torch.float32 and tuple(t.shape) == shape and t.device == dev and t.is_contiguous(),
              f"{name} must be a contiguous float32 tensor of shape {shape} on {dev}")
    lib = _lib.load()
    code = _DTYPES[Z.dtype]
    with _on(dev) as stream:
        ws = _workspace(lib, code, V, r, N, k, dev)
        dZ = torch.empty_like(Z) if want_dZ else None
        dP = torch.empty_like(P) if want_dP else None
        _lib.check(lib.lrhead_distill_grad(code, V, r, _ptr(P), _ptr(Z), N, _ptr(idx), _ptr(logits), k, temperature,
                                           _ptr(lse), _ptr(grad) if want_dZ else None, _ptr(weight), _ptr(dZ),
                                           _ptr(dP), _ptr(ws), ws.numel(), stream), "lrhead_distill_grad")
    return dZ, dP


def _no_capture() -> None:
    # Under graph capture autograd's own accumulation nodes may belong to
    # another stream; the process would end, so the call is refused.
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError("distill_loss cannot be captured with gradients; capture distill and distill_grad")


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Z, P, idx, logits, temperature):
        need_dZ = ctx.needs_input_grad[0]
        _no_capture()
        loss, lse, grad = distill(Z, P, idx, logits, temperature=temperature, want_grad=need_dZ)
        ctx.save_for_backward(Z, P, idx, logits, lse, grad)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        _no_capture()
        Z, P, idx, logits, lse, grad = ctx.saved_tensors
        dZ, dP = distill_grad(Z, P, idx, logits, lse, grad, g.to(torch.float32).contiguous(),
                              temperature=ctx.temperature, want_dZ=ctx.needs_input_grad[0],
                              want_dP=ctx.needs_input_grad[1])
        return dZ, dP, None, None, None


def distill_loss(Z: torch.Tensor, P: torch.Tensor, idx: torch.Tensor, logits: torch.Tensor, *,
                 temperature: float = 1.0) -> torch.Tensor:
    """distill()'s loss [N], differentiable in Z and P. The teacher's logits
    get no gradient. Not for graph capture with gradients: capture distill and
    distill_grad."""
    if not (torch.is_grad_enabled() and (Z.requires_grad or P.requires_grad)):
        return distill(Z, P, idx, logits, temperature=temperature, want_grad=False)[0]
    return _Distill.apply(Z, P, idx, logits, float(temperature))
