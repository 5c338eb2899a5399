"""distill_loss under torch's transforms: what it has no derivative for, it
refuses. On the CPU, with a stand-in for the kernels' call."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import rank_lm_head_amd as lr
from rank_lm_head_amd import train


@pytest.fixture
def stub(monkeypatch):
    def distill(Z, P, idx, logits, *, temperature=1.0, want_grad=True):
        n, r = Z.shape
        return torch.zeros(n), torch.zeros(n), torch.zeros(n, r) if want_grad else None
    monkeypatch.setattr(train, "distill", distill)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return torch.randn(3, 16), torch.randn(50, 16), torch.zeros(3, 4, dtype=torch.int32), torch.randn(3, 4)


@pytest.mark.parametrize("which", ["Z", "P", "logits"])
@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(stub, which, grad):
    """A dual tensor does not require a gradient: its tangent must not be dropped."""
    Z, P, idx, t = stub
    if grad:
        P.requires_grad_()
    with fw.dual_level():
        dual = {"Z": Z, "P": P, "logits": t}
        dual[which] = fw.make_dual(dual[which], torch.ones_like(dual[which]))
        with pytest.raises(NotImplementedError, match="forward"):
            lr.distill_loss(dual["Z"], dual["P"], idx, dual["logits"])
        with torch.no_grad(), pytest.raises(NotImplementedError, match="forward"):
            lr.distill_loss(dual["Z"], dual["P"], idx, dual["logits"])
        assert lr.distill_loss(Z.detach(), P.detach(), idx, t).shape == (3,)   # none of it is dual: as ever
    with pytest.raises((NotImplementedError, RuntimeError)):
        torch.func.jvp(lambda z: lr.distill_loss(z, P.detach(), idx, t), (Z,), (torch.ones_like(Z),))


def test_without_tangents_the_loss_comes_through(stub):
    Z, P, idx, t = stub
    assert not lr.distill_loss(Z, P, idx, t).requires_grad
    assert lr.distill_loss(Z.requires_grad_(), P, idx, t).requires_grad


def test_tensors_that_need_gradients_are_checked_first():
    """A CPU tensor is refused as such, with gradients as without."""
    idx, t = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4)
    for Z in (torch.zeros(3, 16), torch.zeros(3, 16, requires_grad=True)):
        with pytest.raises(ValueError, match="device tensor"):
            lr.distill_loss(Z, torch.zeros(50, 16), idx, t)
