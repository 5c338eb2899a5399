"""Python binding of the head's distillation (argument marshalling only).

distill / distill_grad are the two calls of include/lrhead.h; distill_loss
joins them for torch's autograd.
"""
from __future__ import annotations

import torch
from torch.autograd.forward_ad import unpack_dual

from . import _lib
from .head import _DTYPES, _on


def _check(Z, P, idx, logits):
    """(dtype code, N, V, r, k) of a call's inputs."""
    code = _DTYPES.get(Z.dtype)
    if code is None or P.dtype != Z.dtype:
        raise ValueError(f"Z and P must share a supported dtype (bfloat16 or float32), not {Z.dtype} and {P.dtype}")
    if not Z.is_cuda:
        raise ValueError("Z must be a device tensor")
    if Z.dim() != 2 or P.dim() != 2 or P.shape[1] != Z.shape[1]:
        raise ValueError(f"Z must be (N, r) and P (V, r), not {tuple(Z.shape)} and {tuple(P.shape)}")
    N, r = Z.shape
    if idx.dtype != torch.int32 or logits.dtype != torch.float32:
        raise ValueError(f"idx must be int32 and logits float32, not {idx.dtype} and {logits.dtype}")
    if idx.dim() != 2 or idx.shape[0] != N or logits.shape != idx.shape:
        raise ValueError(f"idx and logits must be ({N}, k), not {tuple(idx.shape)} and {tuple(logits.shape)}")
    dev = Z.device
    for t in (Z, P, idx, logits):
        if t.device != dev or not t.is_contiguous():
            raise ValueError(f"Z, P, idx and logits must be contiguous on {dev}")
    return code, N, P.shape[0], r, idx.shape[1]


def _workspace(lib, code, V, r, N, k, device):
    n = lib.lrhead_distill_workspace_bytes(code, V, r, N, k)
    # without sizes that can be, the call itself says why
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def distill(Z: torch.Tensor, P: torch.Tensor, idx: torch.Tensor, logits: torch.Tensor, *, temperature: float = 1.0,
            want_grad: bool = True):
    """The loss of the rows Z ([N, r]) under the head P ([V, r]) against a
    teacher's top logits (idx int32 and logits float32, [N, k], as
    Head.full_topk returns them; an id outside [0, V), or a logit that is NaN
    or -inf, marks an empty place):
    (loss [N], lse [N], dloss/dZ [N, r] or None), float32. See lrhead_distill
    in include/lrhead.h."""
    code, N, V, r, k = _check(Z, P, idx, logits)
    lib = _lib.load()
    dev = Z.device
    with _on(dev) as stream:
        ws = _workspace(lib, code, V, r, N, k, dev)
        loss = torch.empty(N, dtype=torch.float32, device=dev)
        lse = torch.empty(N, dtype=torch.float32, device=dev)
        grad = torch.empty((N, r), dtype=torch.float32, device=dev) if want_grad else None
        rc = lib.lrhead_distill(code, V, r, P.data_ptr(), Z.data_ptr(), N, idx.data_ptr(), logits.data_ptr(), k,
                                temperature, loss.data_ptr(), lse.data_ptr(), None if grad is None else grad.data_ptr(),
                                None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), stream)
        if rc:
            _lib.check(rc, "lrhead_distill")
    return loss, lse, grad


def distill_grad(Z: torch.Tensor, P: torch.Tensor, idx: torch.Tensor, logits: torch.Tensor, lse: torch.Tensor,
                 grad: torch.Tensor | None, weight: torch.Tensor | None = None, *, temperature: float = 1.0,
                 want_dZ: bool = True, want_dP: bool = True):
    """The gradients of sum(weight * loss): (dZ [N, r] or None, dP [V, r] or
    None) in Z's dtype, from lse and grad of distill() on the same inputs
    (grad may be None without dZ). weight: [N] float32, None for ones. See
    lrhead_distill_grad in include/lrhead.h."""
    code, N, V, r, k = _check(Z, P, idx, logits)
    dev = Z.device
    if want_dZ and grad is None:
        raise ValueError("dZ needs the grad of distill()")
    for name, t, shape in (("lse", lse, (N,)), ("grad", grad if want_dZ else None, (N, r)), ("weight", weight, (N,))):
        if t is not None and (t.dtype != torch.float32 or t.shape != shape or t.device != dev
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 tensor of shape {shape} on {dev}")
    lib = _lib.load()
    with _on(dev) as stream:
        ws = _workspace(lib, code, V, r, N, k, dev)
        dZ = torch.empty_like(Z) if want_dZ else None
        dP = torch.empty_like(P) if want_dP else None
        rc = lib.lrhead_distill_grad(code, V, r, P.data_ptr(), Z.data_ptr(), N, idx.data_ptr(), logits.data_ptr(), k,
                                     temperature, lse.data_ptr(), grad.data_ptr() if want_dZ else None,
                                     None if weight is None else weight.data_ptr(),
                                     None if dZ is None else dZ.data_ptr(), None if dP is None else dP.data_ptr(),
                                     None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), stream)
        if rc:
            _lib.check(rc, "lrhead_distill_grad")
    return dZ, dP


def _no_capture(device) -> None:
    # Under graph capture autograd's own accumulation nodes may belong to
    # another stream; the process would end, so the call is refused.
    with _on(device):
        capturing = torch.cuda.is_current_stream_capturing()
    if capturing:
        raise RuntimeError("distill_loss cannot be captured with gradients; capture distill and distill_grad")


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Z, P, idx, logits, temperature):
        need_dZ = ctx.needs_input_grad[0]
        if Z.is_cuda:   # else distill() says so
            _no_capture(Z.device)
        loss, lse, grad = distill(Z, P, idx, logits, temperature=temperature, want_grad=need_dZ)
        ctx.save_for_backward(Z, P, idx, logits, lse, grad)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        Z, P, idx, logits, lse, grad = ctx.saved_tensors
        _no_capture(Z.device)
        dZ, dP = distill_grad(Z, P, idx, logits, lse, grad, g.to(torch.float32).contiguous(),
                              temperature=ctx.temperature, want_dZ=ctx.needs_input_grad[0],
                              want_dP=ctx.needs_input_grad[1])
        return dZ, dP, None, None, None


def distill_loss(Z: torch.Tensor, P: torch.Tensor, idx: torch.Tensor, logits: torch.Tensor, *,
                 temperature: float = 1.0) -> torch.Tensor:
    """distill()'s loss [N], differentiable in Z and P (backwards only:
    tensors with a forward-mode tangent are refused). The teacher's logits
    get no gradient. Not for graph capture with gradients: capture distill and
    distill_grad."""
    # a tangent does not show in requires_grad, and no_grad does not end it
    if any(unpack_dual(x).tangent is not None for x in (Z, P, logits)):
        raise NotImplementedError("distill_loss has no forward-mode derivative")
    if not (torch.is_grad_enabled() and (Z.requires_grad or P.requires_grad)):
        return distill(Z, P, idx, logits, temperature=temperature, want_grad=False)[0]
    return _Distill.apply(Z, P, idx, logits, float(temperature))
