"""Beam selection over candidate lists longer than a wave, against the definition in 64 bits."""
import pytest
import torch

from test_beam import DEV, NEG, check, draw


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("B,m,n,nb", [(3, 4, 65, 5), (2, 5, 900, 17), (3, 2, 5001, 40), (1, 3, 70000, 8)])
def test_lists_longer_than_a_wave(B, m, n, nb, dt):
    x, score, ids = draw(B, m, n, dt, seed=n, lists=True)
    ids[0, 0, ::3] = -1              # empty slots by id
    x[0, 1, 5:] = float("nan")       # and by logit
    x[B - 1, m - 1, ::2] = NEG
    ids[B - 1, 0] = -1               # a beam with none
    ended = torch.zeros(B, m, dtype=torch.bool, device=DEV)
    ended[0, m - 1] = True
    check(x, score, nb, idx=ids)
    check(x, score, nb, idx=ids, ended=ended, end_id=3)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_best_of_a_list_that_has_no_id(dt):
    """The largest logits belong to empty slots: they are no candidates and have no share of the sum."""
    x, score, ids = draw(2, 2, 3000, dt, seed=8, lists=True)
    x[:, :, 100:140] += 30
    ids[:, :, 100:140] = -1
    s, beam, token = check(x, score, 6, idx=ids)
    assert bool((token >= 0).all())
