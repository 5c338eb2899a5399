"""Sampling against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import rank_lm_head_amd as lr
from sampling_ref import BORDER, draw, weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
LOW = {"bf16": float(torch.finfo(torch.bfloat16).min), "fp32": float(torch.finfo(torch.float32).min)}


def values(kind, B, n, dtype, rng):
    """[B, n] logits as float32 that the type holds exactly."""
    if kind == "noise":
        x = rng.standard_normal((B, n)) * 2.5
    elif kind == "model":
        x = rng.standard_normal((B, n)) * 2
        for b in range(B):
            top = min(n, 100)
            at = rng.permutation(n)[:top]
            x[b, at] = 18 - 2 * np.log1p(np.arange(top)) + 0.1 * rng.standard_normal(top)
    elif kind == "flat":
        x = rng.standard_normal((B, n)) * 0.01
    elif kind == "same":
        x = np.full((B, n), 1.5)
    elif kind == "ties":
        x = rng.integers(0, 4, (B, n)) * 1.0
    elif kind == "rising":
        x = np.sort(rng.standard_normal((B, n)) * 3, axis=1)
    elif kind == "falling":
        x = -np.sort(rng.standard_normal((B, n)) * 3, axis=1)
    elif kind == "masked":
        x = rng.standard_normal((B, n)) * 2.5
        x[rng.random((B, n)) < 0.5] = -np.inf
        x[rng.random((B, n)) < 0.05] = np.nan
        x[0] = -np.inf
        if B > 1:
            x[1] = np.nan
        if B > 2:
            x[2, :] = -np.inf
            x[2, n // 2] = -5.0
    elif kind == "lowest":
        x = rng.standard_normal((B, n)) * 2.5
        x[rng.random((B, n)) < 0.9] = LOW[dtype]
        x[0] = LOW[dtype]
    elif kind == "infinite":
        x = rng.standard_normal((B, n)) * 2.5
        x[:, n // 3] = np.inf
    elif kind == "wide":
        x = rng.standard_normal((B, n)) * 1e30
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    return t


def check(x, u, got, settings, ids=None, probs=None):
    """got: (token, prob) of rows x; settings: one dict or one per row."""
    token, prob = (t.cpu().numpy() for t in got)
    ref = x.float().double().numpy()
    undecided = 0
    for b in range(len(ref)):
        how = settings[b] if isinstance(settings, list) else settings
        row = ref[b].copy()
        if ids is not None:
            row[ids[b].numpy() < 0] = -np.inf
        w, near = weights(row, **how)
        at, near2 = draw(w, u[b])
        if min(near, near2) < BORDER:
            undecided += 1
            continue
        want = -1 if at < 0 else at if ids is None else int(ids[b, at])
        assert token[b] == want, (b, how, token[b], want, near, near2)
        p = 0.0 if at < 0 else w[at] / w.sum()
        # the result's rounding to fp32, and sums off by BORDER
        assert abs(prob[b] - p) <= p * (2.0 ** -24 + 1e-9) + 1e-30, (b, how, prob[b], p)
        if probs is not None:
            q = w / w.sum() if at >= 0 else w
            assert np.all(np.abs(probs[b].cpu().numpy() - q) <= q * (2.0 ** -24 + 1e-9) + 2.0 ** -50), (b, how)
    return undecided


SETTINGS = {
    "whole": dict(),
    "greedy": dict(T=0.0),
    "hot": dict(T=5.0),
    "cold": dict(T=1e-3),
    "k1": dict(k=1),
    "k20": dict(T=0.6, k=20),
    "k20p": dict(T=0.6, k=20, p=0.95),
    "k300": dict(T=1.2, k=300, p=0.97, m=0.01),
    "k5000": dict(k=5000, p=0.9),
    "p90": dict(T=0.8, p=0.9),
    "p999": dict(p=0.999),
    "p0": dict(p=0.0),
    "p1e-6": dict(p=1e-6),
    "p1-": dict(p=1 - 2.0 ** -24, T=1.5),
    "m05": dict(m=0.05),
    "m1": dict(m=1.0),
    "m1e-9": dict(m=1e-9, T=2.0),
    "all": dict(T=0.9, k=100, p=0.9, m=0.02),
    "Tinf": dict(T=float("inf"), k=700),
    "Tinf_whole": dict(T=float("inf")),
}


def settings_args(how):
    return dict(temperature=how.get("T", 1.0), top_k=how.get("k", 0), top_p=how.get("p", 1.0), min_p=how.get("m", 0.0))


@pytest.mark.parametrize("how", SETTINGS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_every_setting(how, dtype):
    rng = np.random.default_rng(sorted(SETTINGS).index(how) * 2 + (dtype == "bf16"))
    undecided = total = 0
    for kind, B, n in [("noise", 5, 1), ("noise", 6, 2), ("model", 7, 64), ("noise", 4, 65), ("masked", 6, 300),
                       ("ties", 4, 2048), ("model", 5, 2049), ("noise", 3, 5003), ("same", 3, 9000), ("model", 3, 32003),
                       ("noise", 2, 70000), ("flat", 2, 30000), ("rising", 2, 20011), ("falling", 2, 20011),
                       ("lowest", 4, 12345), ("infinite", 2, 4100), ("wide", 2, 3000)]:
        x = values(kind, B, n, dtype, rng)
        u = torch.from_numpy(rng.random(B).astype(np.float32))
        print(f"[run] {how} {dtype} {kind} {B}x{n}", flush=True)
        token, prob, _ = lr.sample(x.to(DEV), u.to(DEV), **settings_args(SETTINGS[how]))
        undecided += check(x, u.numpy(), (token, prob), SETTINGS[how])
        total += B
    # rows of few distinct sums lie on borders by themselves, and the tail's sums crowd around a top_p next to 1
    assert undecided <= total // (2 if how == "p1-" else 8)


@pytest.mark.parametrize("kind", ["model", "noise", "masked"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_vocabulary_with_a_setting_for_each_row(kind, dtype):
    rng = np.random.default_rng(7)
    names = list(SETTINGS)
    B, n = len(names), 151936
    x = values(kind, B, n, dtype, rng)
    u = torch.from_numpy(rng.random(B).astype(np.float32))
    how = [SETTINGS[k] for k in names]
    col = lambda key, other, dt: torch.tensor([h.get(key, other) for h in how], dtype=dt, device=DEV)  # noqa: E731
    f = torch.float32
    token, prob, none = lr.sample(x.to(DEV), u.to(DEV), temperature=col("T", 1.0, f), top_k=col("k", 0, torch.int32),
                                  top_p=col("p", 1.0, f), min_p=col("m", 0.0, f))
    assert none is None
    assert check(x, u.numpy(), (token, prob), how) <= 2


def test_larger_rows():
    """More groups of columns than a wave holds, and a row's columns past 2^20."""
    rng = np.random.default_rng(8)
    n = (1 << 20) + 77
    x = values("noise", 2, n, "bf16", rng)
    u = torch.tensor([0.3, 0.9])
    for name in ("whole", "k20p", "k300", "p90", "m05"):
        got = lr.sample(x.to(DEV), u.to(DEV), **settings_args(SETTINGS[name]))[:2]
        check(x, u.numpy(), got, SETTINGS[name])


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_candidate_lists(n, dtype):
    rng = np.random.default_rng(n)
    B = 37
    for name in ("whole", "k20p", "p90", "m05", "greedy", "all"):
        x = values("noise", B, n, dtype, rng)
        x[3] = float("-inf")
        ids = torch.from_numpy(np.stack([rng.permutation(1000)[:n] for _ in range(B)]).astype(np.int32))
        ids[torch.from_numpy(rng.random((B, n)) < 0.2)] = -1
        ids[5] = -1
        u = torch.from_numpy(rng.random(B).astype(np.float32))
        token, prob, probs = lr.sample(x.to(DEV), u.to(DEV), idx=ids.to(DEV), want_probs=True,
                                       **settings_args(SETTINGS[name]))
        check(x, u.numpy(), (token, prob), SETTINGS[name], ids, probs)
        assert token[5] == -1 and token[3] == -1 and probs[5].abs().sum() == 0


def test_long_lists_with_ids():
    rng = np.random.default_rng(1)
    B, n = 6, 9001
    x = values("noise", B, n, "fp32", rng)
    ids = torch.from_numpy(rng.integers(0, 10 ** 6, (B, n)).astype(np.int32))
    ids[torch.from_numpy(rng.random((B, n)) < 0.3)] = -7
    u = torch.from_numpy(rng.random(B).astype(np.float32))
    for name in ("whole", "k20p", "p90", "p999", "k5000", "m05"):
        got = lr.sample(x.to(DEV), u.to(DEV), idx=ids.to(DEV), **settings_args(SETTINGS[name]))[:2]
        check(x, u.numpy(), got, SETTINGS[name], ids)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,ld,first", [(2050, 2051, 1), (64, 67, 3), (30000, 30001, 1), (151, 500, 7)])
def test_rows_of_a_wider_matrix(n, ld, first, dtype):
    """Rows that begin at any element: a slice of a larger tensor's columns."""
    rng = np.random.default_rng(n)
    x = values("noise", 5, ld, dtype, rng)
    u = torch.from_numpy(rng.random(5).astype(np.float32))
    view = x.to(DEV)[:, first:first + n] if first + n <= ld else x.to(DEV)[:, :n]
    cols = view.cpu()
    for name in ("whole", "k20p", "p90"):
        got = lr.sample(view, u.to(DEV), **settings_args(SETTINGS[name]))[:2]
        check(cols, u.numpy(), got, SETTINGS[name])


@pytest.mark.parametrize("n", [5, 64, 65, 30000])
def test_the_ends_of_u(n):
    """u of 0, below 0, NaN: the first kept column; of 1 and above: the last of a weight above 0."""
    rng = np.random.default_rng(n)
    us = torch.tensor([0.0, -3.0, float("nan"), 1 - 2.0 ** -24, 1.0, 2.0, float("inf")])
    x = values("noise", 1, n, "fp32", rng).repeat(len(us), 1)
    x[:, 0] = float("-inf")
    x[:, n - 1] = -3e38
    for name in ("whole", "p90", "k20"):
        token = lr.sample(x.to(DEV), us.to(DEV), **settings_args(SETTINGS[name]))[0].cpu()
        w, _ = weights(x[0].double().numpy(), **SETTINGS[name])
        some = np.flatnonzero(w > 2.0 ** -40)
        assert (token[:3] == int(some[0])).all()
        assert (token[4:] == token[4]).all() and int(token[4]) == int(some[-1])


def test_minus_zero_ties_with_zero():
    x = torch.full((2, 100), -9.0)
    x[:, 7], x[:, 3] = 0.0, -0.0
    token = lr.sample(x.to(DEV), torch.tensor([0.5, 0.5], device=DEV), top_k=1)[0]
    assert token.tolist() == [3, 3]


@pytest.mark.parametrize("kind,n,how", [
    ("same", 20000, dict(p=0.5)), ("same", 20000, dict(k=7777)), ("same", 100000, dict(k=100000 - 1)),
    ("same", 9000, dict()), ("same", 9000, dict(m=1.0)), ("ties", 50000, dict(k=20001)), ("ties", 50000, dict(p=0.3)),
])
def test_long_ties(kind, n, how):
    """Ties at the border go to the lower columns, however many there are: with u near 1 the last kept one shows."""
    rng = np.random.default_rng(5)
    x = values(kind, 1, n, "bf16", rng)
    us = torch.tensor([0.1, 0.5, 0.9, 1 - 2.0 ** -24])
    x = x.repeat(len(us), 1)
    got = lr.sample(x.to(DEV), us.to(DEV), **settings_args(how))[:2]
    token = got[0].cpu().numpy()
    w, _ = weights(x[0].double().numpy(), **how)
    c = np.cumsum(w) / w.sum()
    for t, u in zip(token, us.double().numpy()):
        assert w[t] > 0 and c[t] >= u - 1e-9 and (t == 0 or c[t - 1] <= u + 1e-9)


def test_a_group_full_of_the_best():
    """More of the best columns under one maximum than the bound expects, and more than the list holds."""
    rng = np.random.default_rng(2)
    for n, lo, hi in [(40000, 512, 768), (60000, 10000, 17000)]:
        x = values("noise", 3, n, "fp32", rng)
        x[:, lo:hi] += 40
        u = torch.tensor([0.2, 0.5, 0.97])
        for how in (dict(k=200), dict(k=40, p=0.9), dict(p=0.95), dict(k=6000), dict(k=5500, p=0.99, m=1e-4), dict(m=1e-3)):
            got = lr.sample(x.to(DEV), u.to(DEV), **settings_args(how))[:2]
            check(x, u.numpy(), got, how)


def test_frequencies():
    """Over an even grid of u, tokens come as often as their probability says, to one grid step a column."""
    rng = np.random.default_rng(3)
    m = 20000
    u = ((torch.arange(m) + 0.5) / m).float()
    for n in (40, 500):
        row = values("noise", 1, n, "fp32", rng)
        token = lr.sample(row.to(DEV).expand(m, n).contiguous(), u.to(DEV), temperature=1.3, top_p=0.97)[0].cpu().numpy()
        w, _ = weights(row[0].double().numpy(), T=1.3, p=0.97)
        assert np.abs(np.bincount(token, minlength=n) / m - w / w.sum()).max() <= 1.01 / m


def test_results_do_not_vary_and_workspaces_need_no_clearing():
    rng = np.random.default_rng(4)
    x = values("noise", 64, 50000, "bf16", rng).to(DEV)
    u = torch.from_numpy(rng.random(64).astype(np.float32)).to(DEV)
    how = dict(temperature=1.1, top_p=0.93)
    first = lr.sample(x, u, **how)
    for _ in range(3):
        lr.sample(x.flip(0).contiguous(), u, top_k=3)
        again = lr.sample(x, u, **how)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_another_stream_and_a_captured_call():
    rng = np.random.default_rng(6)
    x = values("model", 9, 30000, "fp32", rng)
    xs, u = x.to(DEV), torch.from_numpy(rng.random(9).astype(np.float32)).to(DEV)
    how = dict(T=0.9, p=0.9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = lr.sample(xs, u, **settings_args(how))[:2]
    side.synchronize()
    check(x, u.cpu().numpy(), got, how)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token, prob, _ = lr.sample(xs, u, **settings_args(how))
    for i in range(4):
        new = values("model", 9, 30000, "fp32", rng)
        xs.copy_(new)
        u.copy_(torch.from_numpy(rng.random(9).astype(np.float32)))
        graph.replay()
        lr.sample(xs, u, top_k=5)     # the program's own work between replays
        torch.cuda.synchronize()
        check(new, u.cpu().numpy(), (token, prob), how)


def test_no_rows():
    token, prob, probs = lr.sample(torch.zeros(0, 32, device=DEV), torch.zeros(0, device=DEV), want_probs=True)
    assert token.shape == (0,) and prob.shape == (0,) and probs.shape == (0, 32)
    assert lr.sample(torch.zeros(0, 3200, device=DEV), torch.zeros(0, device=DEV))[0].shape == (0,)


def of_each_row(hows):
    col = lambda key, other, dt: torch.tensor([h.get(key, other) for h in hows], dtype=dt, device=DEV)  # noqa: E731
    f = torch.float32
    return dict(temperature=col("T", 1.0, f), top_k=col("k", 0, torch.int32), top_p=col("p", 1.0, f),
                min_p=col("m", 0.0, f))


@pytest.mark.parametrize("kind", ["noise", "model", "masked", "rising", "wide"])
@pytest.mark.parametrize("n", [2049, 5000, 20001])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_more_kept_columns_than_groups_of_columns(n, kind, dtype):
    rng = np.random.default_rng(17)
    hows = [dict(k=40), dict(k=200, p=0.98, T=1.2), dict(k=900), dict(p=0.9, T=0.7), dict(p=0.98, m=0.02),
            dict(k=1023, m=0.01), dict(k=1024), dict(k=2049)]
    B = len(hows)
    x = values(kind, B, n, dtype, rng)
    u = torch.from_numpy(rng.random(B).astype(np.float32))
    got = lr.sample(x.to(DEV), u.to(DEV), **of_each_row(hows))[:2]
    assert check(x, u.numpy(), got, hows) <= 2


@pytest.mark.parametrize("left", [3, 60, 300, 3000])
def test_candidates_in_few_groups_only(left):
    rng = np.random.default_rng(23)
    hows = [dict(k=40), dict(k=500, p=0.95), dict(p=0.9), dict(k=2500)]
    B, n = len(hows), 40003
    x = torch.full((B, n), -float("inf"))
    x[:, n - 10000:n - 10000 + left] = values("noise", B, left, "fp32", rng)
    u = torch.from_numpy(rng.random(B).astype(np.float32))
    got = lr.sample(x.to(DEV), u.to(DEV), **of_each_row(hows))[:2]
    assert check(x, u.numpy(), got, hows) <= 1


@pytest.mark.parametrize("how", ["whole", "k300", "p90", "m05", "greedy"])
def test_the_longest_rows(how):
    """2^24 columns, a token every 2^-24 of the mass: the draw lies where u says to the sums' accuracy."""
    rng = np.random.default_rng(31)
    n, how = 1 << 24, SETTINGS[how]
    x = torch.from_numpy(rng.standard_normal((2, n), dtype=np.float32) * 2.5).to(torch.bfloat16)
    x[1, :n // 2] = -float("inf")
    u = torch.tensor([0.37, 0.9])
    token, prob, _ = lr.sample(x.to(DEV), u.to(DEV), **settings_args(how))
    for b in range(2):
        w, _ = weights(x[b].float().double().numpy(), **how)
        c, t = np.cumsum(w), int(token[b])
        # half a unit of 2^-38 for each weight, on both sides of a border, and 64-bit sums over 2^24 columns; as much
        # again, of 0.9 of the mass, for the border of top_p
        off = 2 * (2 * n * 2.0 ** -39 / c[-1] + 1e-8) / 0.9
        place = float(u[b])
        assert w[t] > 0 and c[t] / c[-1] >= place - off and (c[t] - w[t]) / c[-1] <= place + off
        assert abs(float(prob[b]) - w[t] / c[-1]) <= w[t] / c[-1] * (2.0 ** -24 + off) + 2.0 ** -39 / c[-1]


@pytest.mark.parametrize("kind", ["model", "noise", "flat", "masked", "ties"])
@pytest.mark.parametrize("n,dtype", [(700, "fp32"), (9001, "bf16"), (9001, "fp32"), (40003, "bf16")])
def test_large_batches_give_what_small_ones_do(n, dtype, kind):
    """More rows than compute units, under every setting, against the same rows by themselves; some against the formula."""
    rng = np.random.default_rng(41)
    names = list(SETTINGS)
    B = 20 * len(names)
    hows = [SETTINGS[names[b % len(names)]] for b in range(B)]
    x = values(kind, B, n, dtype, rng)
    u = torch.from_numpy(rng.random(B).astype(np.float32))
    args = of_each_row(hows)
    got = lr.sample(x.to(DEV), u.to(DEV), **args)[:2]
    for b0 in range(0, B, 100):
        part = lr.sample(x[b0:b0 + 100].to(DEV), u[b0:b0 + 100].to(DEV), **{k: v[b0:b0 + 100].clone() for k, v in args.items()})
        for whole, one in zip(got, part):
            assert torch.equal(whole[b0:b0 + 100], one)
    first = len(names)   # a row of each; flat rows and ties lie on borders by themselves
    undecided = check(x[:first], u[:first].numpy(), [t[:first] for t in got], hows[:first])
    assert undecided <= (first // 2 if kind in ("flat", "ties") else 2)


def test_rows_past_32_bits():
    """Rows more than 2^31 elements apart, and settings that read them again."""
    n, ld = 50000, (1 << 31) + 5
    rng = np.random.default_rng(47)
    x = values("noise", 3, n, "bf16", rng)
    big = torch.empty(2 * ld + n, dtype=torch.bfloat16, device=DEV).as_strided((3, n), (ld, 1))
    big.copy_(x.to(DEV))
    u = torch.from_numpy(rng.random(3).astype(np.float32)).to(DEV)
    for how in SETTINGS.values():
        for far, near in zip(lr.sample(big, u, **settings_args(how))[:2], lr.sample(x.to(DEV), u, **settings_args(how))[:2]):
            assert torch.equal(far, near)
