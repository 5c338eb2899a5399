"""Tensors given as `out` are changed in place, and autograd knows it."""
import pytest
import torch

import rank_lm_head_amd as lr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def refuses_backward_after(change, out):
    x = torch.ones(out.shape, device=DEV, requires_grad=True)
    y = (x * out).sum()      # keeps out for x's gradient
    before = out._version
    change()
    assert out._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("N", [3, 700])
def test_embed_grad(N):
    dY, t = torch.ones(N, 8, device=DEV), torch.zeros(N, dtype=torch.int32, device=DEV)
    out = torch.ones(5, 8, device=DEV)
    refuses_backward_after(lambda: lr.embed_grad(dY, t, 5, out=out), out)
    assert (out[0] == 1 + N).all() and (out[1:] == 1).all()
    with torch.inference_mode():   # tensors without a version
        out = torch.ones(5, 8, device=DEV)
        lr.embed_grad(dY, t, 5, out=out)
    assert (out[0] == 1 + N).all()


def test_reorder():
    states = [torch.randn(2, 3, 4, 8, device=DEV), torch.randn(2, 3, 5, device=DEV)]
    parent = torch.tensor([[2, 0], [1, 1]], dtype=torch.int32, device=DEV)
    outs = [torch.zeros(2, 2, 4, 8, device=DEV), torch.zeros(2, 2, 5, device=DEV)]
    refuses_backward_after(lambda: lr.reorder(states, parent, out=outs), outs[1])
    refuses_backward_after(lambda: lr.reorder(states[0], parent, out=outs[0]), outs[0])
    for x, o in zip(states, outs):
        for b in range(2):
            for j in range(2):
                assert torch.equal(o[b, j], x[b, int(parent[b, j])])
    got = lr.reorder(states, parent, out=[None, outs[1]])
    assert torch.equal(got[0], outs[0]) and got[1] is outs[1]
    with torch.inference_mode():
        got = lr.reorder(states[0], parent, out=torch.zeros(2, 2, 4, 8, device=DEV))
    assert torch.equal(got, outs[0])
