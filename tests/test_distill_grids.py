"""Distillation over the grids of large steps, small enough for a check in 64
bits: groups of columns that stream all rows followed by groups that share
them out, shares of many tiles, and shares whose exponents' reference fails.
"""
import pytest
import torch

from test_distill import DEV, check, inputs


@pytest.mark.gpu
@pytest.mark.timeout(300)
@pytest.mark.parametrize("N,V,r,dt,whole", [
    # columns up to `whole` belong to groups that stream all rows, the others to groups that share them out
    (200, 66000, 128, "bf16", 512 * 128),
    (100, 66000, 256, "bf16", 512 * 128),
    (100, 34000, 512, "bf16", 256 * 128),
    (200, 132000, 64, "bf16", 512 * 256),
    (200, 132000, 24, "bf16", 512 * 256),
    (200, 66000, 64, "fp32", 1024 * 64),
    (200, 34000, 256, "fp32", 512 * 64),
])
def test_whole_and_shared_groups_of_columns(N, V, r, dt, whole):
    k = 24
    Z, P, idx, t, w = inputs(N, V, r, k, dt, seed=V + r)
    edge = torch.tensor([whole - 129, whole - 2, whole - 1, whole, whole + 1, whole + 130, V - 1, 0], dtype=torch.int32)
    idx[:, :8] = edge                # on both sides of the last whole group
    idx[:, 8:16] = torch.arange(8, dtype=torch.int32) + whole + 16   # a frequent group of the shared part
    idx[:, 16:20] = torch.arange(4, dtype=torch.int32) + 300         # and one of the whole part
    check(Z, P, idx.contiguous(), t, w, 1.0, dt)


@pytest.mark.gpu
@pytest.mark.timeout(300)
@pytest.mark.parametrize("N,V,r", [
    (1030, 18001, 512),   # 20 tiles a share
    (2050, 20001, 128),   # 10
    (2050, 12001, 32),
    (1030, 9001, 256),
])
def test_shares_of_many_tiles(N, V, r):
    check(*inputs(N, V, r, 12, "bf16", seed=N + r), 1.0, "bf16")


@pytest.mark.gpu
@pytest.mark.timeout(300)
@pytest.mark.parametrize("N,V,r", [
    (20, 132100, 32),    # four waves share a row's tiles (128 rows each); shares of two or three
    (50, 66100, 128),    # two do (64 rows)
    (20, 33100, 304),
    (300, 33100, 64),    # none (64 rows); shares of two or more
    (300, 33100, 128),   # three or more
    (300, 17100, 256),   # 32 rows
    (130, 9100, 512),
])
def test_shares_whose_first_scores_are_low(N, V, r):
    """The exponents' reference, the largest of a share's first 32 scores, is
    passed by far more than 2^60 behind them: the share is done again. Odd
    blocks of 32 tokens lie 64 above even ones, and tiles of 64 or 128 tokens
    begin with an even one; of the tiles of 32, every second does."""
    Z, P, idx, t, w = inputs(N, V, r, 9, "bf16", seed=N + r)
    block = torch.arange(V, device=DEV) // 32
    Z[:, 0] = 8.0
    P[:, 0] = torch.where(block % 2 == 1, 4.0, -4.0).to(P.dtype)
    check(Z, P, idx, t, w, 1.0, "bf16")
    P[:, 0] = torch.where(block == block[-1], 4.0, -4.0).to(P.dtype)   # only the last tile, which the vocabulary ends in
    check(Z, P, idx, t, w, 1.0, "bf16")
