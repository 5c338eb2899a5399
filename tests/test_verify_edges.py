"""Verification at its edges: drafted tokens that the target's settings leave out, u outside [0, 1)."""
import numpy as np
import pytest
import torch

import rank_lm_head_amd as lr
from sampling_ref import weights
from test_sample import DEV, DT, SETTINGS, settings_args, values
from test_verify import check, drafts, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1500, 5000, 40000, 151936])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lists", [False, True])
def test_a_token_behind_a_list_of_exactly_top_k(n, dtype, lists):
    """100 columns above all others and top_k = 100: the drafted tokens are among the others, where p = 0."""
    B, s, k = 3, 2, 100
    x = torch.zeros(B, s + 1, n, dtype=DT[dtype])
    top = torch.arange(k) * (n // k) + 3
    x[:, :, top] = 1.0
    token = torch.tensor([[4, n - 1], [int(top[5]), 0], [int(top[0]), int(top[99])]], dtype=torch.int32)
    u = torch.full((B, s + 1), 0.001)
    u[:, s] = torch.tensor([0.0, 0.5, 1 - 2.0 ** -24])
    args = {}
    if lists:
        args = dict(idx=token[:, :, None].contiguous().to(DEV), probs=torch.full((B, s, 1), 0.5, device=DEV))
    out, count = lr.verify(x.to(DEV), token.to(DEV), u.to(DEV), **args, top_k=k)
    out = out.tolist()
    # p is 1 / 100 for each of the 100; what a refused token leaves out has p = 0 itself
    assert out[0] == [int(top[0]), -1, -1]
    assert out[1] == [int(top[5]), int(top[50]), -1]
    assert out[2] == [int(top[0]), int(top[99]), int(top[99])]
    assert count.tolist() == [1, 2, 3]


@pytest.mark.parametrize("n,dtype", [(3000, "fp32"), (9001, "bf16"), (40003, "fp32")])
def test_tokens_behind_top_k_are_refused(n, dtype):
    """Rows as a model has them, top_k from 66 to 125: the columns next behind top_k, at the least u."""
    rng = np.random.default_rng(n)
    B, s = 60, 3
    x = values("model", B * (s + 1), n, dtype, rng).view(B, s + 1, n)
    ks = 66 + np.arange(B)
    order = np.argsort(-x.float().numpy(), axis=2, kind="stable")
    for behind in (0, 1, 40, 1000):
        token = np.stack([order[b, :s, ks[b] + behind] for b in range(B)]).astype(np.int32)
        for how in (dict(), dict(m=1e-6)):
            out, count = lr.verify(x.to(DEV), torch.from_numpy(token).to(DEV), torch.full((B, s + 1), 1e-4, device=DEV),
                                   **{**settings_args(how), "top_k": torch.from_numpy(ks.astype(np.int32)).to(DEV)})
            assert (count == 1).all()
            for b in range(B):
                w, _ = weights(x[b, 0].float().double().numpy(), k=int(ks[b]), **how)
                assert w[int(out[b, 0])] > 0 and out[b, 0] != int(token[b, 0])


OUTSIDE = [0.0, -0.0, -3.0, -float("inf"), float("nan"), 1.0, 2.0, float("inf")]


@pytest.mark.parametrize("how", ["whole", "greedy", "k20p", "k300", "p90", "p999", "m05"])
@pytest.mark.parametrize("n", [30, 3000, 20011])
@pytest.mark.parametrize("lists", [False, True])
def test_the_ends_of_the_acceptance_numbers(n, how, lists):
    """u below 0 and NaN accept as 0 does: what has weight, and no token left out, masked or outside the vocabulary."""
    rng = np.random.default_rng(n)
    B, s = len(OUTSIDE), 7
    x = values("noise", B * (s + 1), n, "fp32", rng).view(B, s + 1, n)
    x[:, :, 5] = -float("inf")
    order = np.argsort(-x.numpy(), axis=2, kind="stable")
    token, ids, q = drafts(x, 16, rng)
    token[:, 0] = order[:, 0, 0]                       # accepted, unless u q passes p
    for b in range(B):                                 # what must not be accepted, at each of the places behind
        j = 1 + b % 3
        token[b, j] = (5, -1, n)[b % 3]
        ids[b, j, 0] = token[b, j]
    token[:, 4] = order[:, 4, n - 2]                   # the least one
    ids[:, 4, 0] = token[:, 4]
    u = rng.random((B, s + 1)).astype(np.float32)
    u[:, :s] = np.array(OUTSIDE, np.float32)[:, None]
    if not lists:
        ids = q = None
    got = run(x, token, ids, q, u, None, settings_args(SETTINGS[how]))
    held = u.copy()
    held[:, :s] = np.clip(np.nan_to_num(held[:, :s], nan=0.0), 0.0, 1.0)
    # three rows have u = 1, and greedy ones without lists p = q = 1: 1 < 1 lies on the border itself, and refuses
    undecided = 3 if how == "greedy" and not lists else 2
    assert check(x, token, ids, q, held, None, got, SETTINGS[how]) <= undecided
    if undecided == 3:
        assert got[1][5:].tolist() == [1, 1, 1] and np.array_equal(got[0][5:, 0].cpu().numpy(), token[5:, 0])
    for b in range(B):                                 # none passes the place that has no chance
        assert got[1][b] <= 2 + b % 3


@pytest.mark.parametrize("s", [0, 3])
def test_lists_without_a_column_are_refused(s):
    """They are no lists left out: those make the drafted tokens ones of probability 1."""
    x, u = torch.zeros(2, s + 1, 100, device=DEV), torch.zeros(2, s + 1, device=DEV)
    none = torch.zeros(2, s, 0, device=DEV)
    with pytest.raises(ValueError, match="column"):
        lr.verify(x, torch.zeros(2, s, dtype=torch.int32, device=DEV), u, idx=none.int(), probs=none)
