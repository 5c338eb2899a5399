"""Logits of -0 and +0 are the same logit: they tie, whatever group of columns they stand in."""
import numpy as np
import pytest
import torch

import rank_lm_head_amd as lr
from sampling_ref import BORDER
from test_sample import DEV, DT, check, settings_args

pytestmark = pytest.mark.gpu
U = torch.tensor([0.05, 0.3, 0.7, 0.95])


def rows(n, dtype, zeros, rest=-9.0):
    """Four rows of `rest`, with -0 or +0 where `zeros` (column: sign) says."""
    x = torch.full((len(U), n), rest, dtype=DT[dtype])
    for col, sign in zeros.items():
        x[:, col] = sign * 0.0
    return x


def sample(x, how, kept):
    """`kept` columns of equal weights are left in: u is undecided next to a multiple of 1 / kept, and nowhere else."""
    got = lr.sample(x.to(DEV), U.to(DEV), **settings_args(how))[:2]
    at = U.double().numpy() * kept
    assert check(x, U.numpy(), got, how) <= (np.abs(at - np.round(at)) < BORDER * kept).sum()


@pytest.mark.parametrize("how", [dict(k=1), dict(T=0.0), dict(k=3), dict(k=11), dict(k=12)], ids=str)
@pytest.mark.parametrize("n", [40000, 151936])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_lower_columns_come_first_across_groups(n, dtype, how):
    """Twelve groups of columns whose best is -0, and later ones whose best is +0: columns 5, 1005, ... come first."""
    x = rows(n, dtype, {**{5 + 1000 * i: -1.0 for i in range(12)}, **{20000 + 700 * i: 1.0 for i in range(20)}})
    sample(x, how, how.get("k", 1))


@pytest.mark.parametrize("k", [20, 29, 60, 200])
@pytest.mark.parametrize("n", [1500, 5000])
def test_the_lower_columns_come_first_among_few_groups(n, k):
    """More columns than groups of them: sets of columns a step apart give the bound, of -0 first and +0 behind."""
    for dtype in ("bf16", "fp32"):
        sample(rows(n, dtype, {**{c: -1.0 for c in range(3 * k // 2)}, **{c: 1.0 for c in range(3 * k // 2, 4 * k)}}), dict(k=k), k)


# Below, the settings keep what has the largest weight alone.
HIGHEST = [dict(m=1.0), dict(m=2.0), dict(T=0.0, m=1.0), dict(k=5, m=1.0), dict(k=300, m=1.0), dict(p=0.9, m=1.0),
           dict(k=40, p=0.9, m=1.0), dict(T=1e-3, m=1.0)]


@pytest.mark.parametrize("how", HIGHEST, ids=str)
@pytest.mark.parametrize("n", [300, 2048, 2049, 5000, 40000])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_largest_logit_of_minus_zero(n, dtype, how):
    for col in (0, n // 2, n - 1):
        x = rows(n, dtype, {col: -1.0})
        token, prob, _ = lr.sample(x.to(DEV), U.to(DEV), **settings_args(how))
        assert (token == col).all() and (prob == 1).all()


@pytest.mark.parametrize("how", HIGHEST, ids=str)
@pytest.mark.parametrize("n", [2048, 5000, 40000])
def test_a_largest_logit_of_minus_zero_among_lists(n, how):
    """The last row's id is at the end of its array."""
    rng = np.random.default_rng(n)
    ids = torch.from_numpy(rng.integers(0, 10 ** 6, (len(U), n)).astype(np.int32))
    for dtype in ("bf16", "fp32"):
        for col in (1, n - 1):
            x = rows(n, dtype, {col: -1.0})
            token, prob, _ = lr.sample(x.to(DEV), U.to(DEV), idx=ids.to(DEV), **settings_args(how))
            assert torch.equal(token.cpu(), ids[:, col]) and (prob == 1).all()


@pytest.mark.parametrize("how", HIGHEST[:2] + [dict(k=300, m=1.0), dict(p=0.999, m=1.0)], ids=str)
@pytest.mark.parametrize("n", [2048, 5000, 40000])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_zeros_of_both_signs_weigh_the_same(n, dtype, how):
    signs = {3: -1.0, n // 2: 1.0, n - 2: -1.0}
    sample(rows(n, dtype, signs), how, 3)
    sample(rows(n, dtype, {c: -s for c, s in signs.items()}), how, 3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_of_zeros_alone(dtype):
    rng = np.random.default_rng(3)
    n = 9001
    x = torch.from_numpy(np.where(rng.random((len(U), n)) < 0.5, 0.0, -0.0).astype(np.float32)).to(DT[dtype])
    for how in (dict(k=7), dict(k=100), dict(k=3000), dict(m=1.0), dict(p=0.5), dict(k=500, p=0.3, m=1.0), dict()):
        got = [t.cpu() for t in lr.sample(x.to(DEV), U.to(DEV), **settings_args(how))[:2]]
        same = [t.cpu() for t in lr.sample(torch.zeros(len(U), n, dtype=DT[dtype], device=DEV), U.to(DEV), **settings_args(how))[:2]]
        assert torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])


@pytest.mark.parametrize("how", HIGHEST, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_verification_of_a_largest_logit_of_minus_zero(dtype, how):
    n = 5000
    x = rows(n, dtype, {77: -1.0}).view(2, 2, n).to(DEV)
    token = torch.tensor([[77], [78]], dtype=torch.int32, device=DEV)
    out, count = lr.verify(x, token, torch.full((2, 2), 0.5, device=DEV), **settings_args(how))
    assert out.tolist() == [[77, 77], [77, -1]] and count.tolist() == [2, 1]
