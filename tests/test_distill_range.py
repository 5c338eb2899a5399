"""Distillation at the ends of the numbers' range, against the definition in
64 bits (the bounds of tests/test_distill.py)."""
import pytest
import torch

from test_distill import check, inputs


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [0.5, 2.0 ** -10])
@pytest.mark.parametrize("N", [20, 200])
def test_teacher_logits_whose_quotient_by_the_temperature_has_no_place_in_fp32(N, T, dt):
    """Logits at the type's lowest value are places like any others, whatever T is."""
    Z, P, idx, t, w = inputs(N, 900, 64, 6, dt, seed=N, T=T)
    low = torch.finfo(torch.float32).min
    t[0] = low                       # all alike: the same share for each
    t[1, :3] = low                   # none but the others
    t[2] = -low
    t[3, 2:4] = -low                 # none but these two
    t[4, 1:] = low / 2               # one place far above the others, which are far below zero
    t[5] = low / 2
    t[5, 1] = float("-inf")          # empty
    t[6, 0], t[6, 1] = low, -low     # further apart than the type can say
    Z, w = (Z.float() * T).to(Z.dtype), w * T
    loss, lse, grad, dZ, dP = check(Z, P, idx, t, w, T, dt)
    assert bool(torch.isfinite(loss).all()) and bool(grad[0].any()) and bool(grad[2].any())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [20, 200])
@pytest.mark.parametrize("T,w_size,z_size,p_size", [
    (1.0, 1e20, 1.0, 1.0), (1.0, 1e25, 1.0, 1.0), (1e-20, 1.0, 1e-10, 1e-10), (1e-5, 1e18, 1e-5, 1.0),
    (1.0, 1e-30, 1.0, 1.0), (1e20, 1.0, 1e10, 1e10), (64.0, 1.0, 8.0, 8.0),
])
def test_weights_of_any_size(T, w_size, z_size, p_size, N, dt):
    """|w| / T from below the smallest normal number to far above 2^64."""
    Z, P, idx, t, w = inputs(N, 900, 64, 6, dt, seed=N)
    Z, P = (Z.float() * z_size).to(Z.dtype), (P.float() * p_size).to(P.dtype)
    loss, lse, grad, dZ, dP = check(Z, P, idx, t * T, w * w_size, T, dt)
    assert bool(torch.isfinite(dP).all())
