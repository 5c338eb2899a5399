"""Verification of drafted tokens against its definition in 64 bits."""
import numpy as np
import pytest
import torch

import rank_lm_head_amd as lr
from sampling_ref import BORDER, verify, weights
from test_sample import DEV, SETTINGS, settings_args, values

pytestmark = pytest.mark.gpu


def drafts(x, k, rng, noise=0.7, T=1.0):
    """Candidate lists of a drafter that sees the target through noise, and tokens drawn from them: [B, s, ...]."""
    B, m, n = x.shape
    s = m - 1
    guess = np.nan_to_num(x[:, :s].float().double().numpy(), nan=-np.inf, posinf=50.0) + noise * rng.standard_normal((B, s, n))
    ids = np.argsort(-guess, axis=2, kind="stable")[:, :, :k].astype(np.int32)
    top = np.take_along_axis(guess, ids.astype(np.int64), 2)
    top = np.where(top > -np.inf, top, -1e30)
    q = np.exp((top - top.max(2, keepdims=True)) / T)
    q = (q / q.sum(2, keepdims=True)).astype(np.float32)
    token = np.zeros((B, s), np.int32)
    for b in range(B):
        for j in range(s):
            token[b, j] = ids[b, j, rng.choice(ids.shape[2], p=q[b, j].astype(np.float64) / q[b, j].sum(dtype=np.float64))]
    return token, ids, q


def run(x, token, ids, q, u, length, how):
    on = lambda t: None if t is None else torch.from_numpy(t).to(DEV)  # noqa: E731
    return lr.verify(x.to(DEV), on(token), on(u), idx=on(ids), probs=on(q), length=on(length), **how)


def check(x, token, ids, q, u, length, got, settings):
    out, count = (t.cpu().numpy() for t in got)
    ref = x.float().double().numpy()
    undecided = 0
    for b in range(len(ref)):
        how = settings[b] if isinstance(settings, list) else settings
        s = token.shape[1] if length is None else int(min(max(length[b], 0), token.shape[1]))
        pick = np.concatenate([u[b, :s], u[b, -1:]])
        want, near = verify(ref[b, :s + 1], token[b, :s], None if ids is None else ids[b], None if q is None else q[b],
                            pick, how)
        if near < BORDER:
            undecided += 1
            continue
        assert count[b] == len(want), (b, how, out[b], want, near)
        assert out[b].tolist() == want + [-1] * (out.shape[1] - len(want)), (b, how, out[b], want, near)
    return undecided


@pytest.mark.parametrize("how", ["whole", "greedy", "cold", "k20", "k20p", "k300", "k5000", "p90", "p999", "p0", "m05", "all",
                                 "Tinf"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_every_setting(how, dtype):
    rng = np.random.default_rng(sorted(SETTINGS).index(how) * 2 + (dtype == "bf16"))
    undecided = total = 0
    for kind, B, s, n, k in [("model", 7, 3, 2000, 8), ("noise", 5, 4, 30, 16), ("model", 3, 5, 20011, 32),
                             ("noise", 4, 2, 5000, 64), ("masked", 3, 2, 700, 4), ("noise", 9, 1, 1, 1),
                             ("lowest", 3, 2, 3001, 9), ("flat", 2, 2, 9000, 64), ("same", 2, 2, 300, 33)]:
        x = values(kind, B * (s + 1), n, dtype, rng).view(B, s + 1, n)
        token, ids, q = drafts(x, min(k, n), rng)
        u = rng.random((B, s + 1)).astype(np.float32)
        print(f"[run] {how} {dtype} {kind} {B}x{s}x{n}", flush=True)
        got = run(x, token, ids, q, u, None, settings_args(SETTINGS[how]))
        undecided += check(x, token, ids, q, u, None, got, SETTINGS[how])
        total += B
    assert undecided <= total // 3      # cold, flat and equal rows often have nothing left of p - q but roundings


def test_a_batch_with_settings_and_lengths_of_its_own():
    rng = np.random.default_rng(11)
    names = list(SETTINGS)
    B, s, n = len(names), 7, 32003
    x = values("model", B * (s + 1), n, "bf16", rng).view(B, s + 1, n)
    token, ids, q = drafts(x, 32, rng)
    u = rng.random((B, s + 1)).astype(np.float32)
    length = rng.integers(-1, s + 3, B).astype(np.int32)     # held to [0, s]
    how = [SETTINGS[k] for k in names]
    col = lambda key, other, dt: torch.tensor([h.get(key, other) for h in how], dtype=dt, device=DEV)  # noqa: E731
    f = torch.float32
    args = dict(temperature=col("T", 1.0, f), top_k=col("k", 0, torch.int32), top_p=col("p", 1.0, f),
                min_p=col("m", 0.0, f))
    got = run(x, token, ids, q, u, length, args)
    assert check(x, token, ids, q, u, length, got, how) <= 4
    # rows behind the last drafted token are not looked at
    y = x.clone()
    for b in range(B):
        y[b, int(min(max(length[b], 0), s)) + 1:] = float("nan")
    again = run(y, token, ids, q, u, length, args)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("how", ["whole", "greedy", "k20p", "p90"])
def test_greedy_drafts_without_lists(how):
    rng = np.random.default_rng(12)
    B, s, n = 12, 3, 4001
    x = values("model", B * (s + 1), n, "fp32", rng).view(B, s + 1, n)
    token = x[:, :s].argmax(2).int().numpy()
    token[rng.random((B, s)) < 0.3] = 5
    token[0, 0], token[1, 0], token[2, 1] = -1, n, 2 ** 31 - 1       # no tokens of the vocabulary: never accepted
    u = rng.random((B, s + 1)).astype(np.float32)
    got = run(x, token, None, None, u, None, settings_args(SETTINGS[how]))
    assert check(x, token, None, None, u, None, got, SETTINGS[how]) <= 3
    assert got[1][0] == 1 and got[1][1] == 1 and got[1][2] <= 2


def test_lists_with_repeated_missing_and_bad_entries():
    rng = np.random.default_rng(13)
    B, s, n, k = 40, 2, 3000, 12
    x = values("model", B * (s + 1), n, "fp32", rng).view(B, s + 1, n)
    token, ids, q = drafts(x, k, rng)
    ids[:, :, 3] = ids[:, :, 1]                   # twice the same: their probabilities add up
    ids[:, :, 5] = -1
    ids[:, :, 6] = n + 3
    q[:, :, 7] = np.nan
    q[:, :, 8] = -0.5
    u = rng.random((B, s + 1)).astype(np.float32)
    for how in ("whole", "p90", "k20p", "k300"):
        got = run(x, token, ids, q, u, None, settings_args(SETTINGS[how]))
        assert check(x, token, ids, q, u, None, got, SETTINGS[how]) <= 4


@pytest.mark.parametrize("n", [8, 6000])
def test_a_draft_of_the_target_itself_is_accepted(n):
    """q = p up to its rounding to fp32 (half a unit of 2^-24 of it): u below 1 - 2^-23 accepts; one of 1 - 2^-24 may not."""
    rng = np.random.default_rng(14)
    B, s = 5, 3
    x = torch.full((B, s + 1, n), float("-inf"))
    x[:, :, :8] = values("noise", B * (s + 1), 8, "fp32", rng).view(B, s + 1, 8)
    q = torch.softmax(x[:, :s, :8].double(), 2).float().numpy()
    ids = np.broadcast_to(np.arange(8, dtype=np.int32), (B, s, 8)).copy()
    token = rng.integers(0, 8, (B, s)).astype(np.int32)
    u = np.full((B, s + 1), 1 - 2.0 ** -22, np.float32)
    out, count = run(x, token, ids, q, u, None, {})
    assert (count == s + 1).all() and torch.equal(out[:, :s].cpu(), torch.from_numpy(token))


@pytest.mark.parametrize("n", [20, 5000])
def test_a_list_that_covers_the_target_leaves_the_target(n):
    """max(0, p - q) without mass: the draw is from p."""
    x = torch.full((3, 2, n), float("-inf"))
    x[:, :, 2:6] = torch.tensor([1.0, 2.0, 0.5, 1.5])
    ids = np.broadcast_to(np.arange(2, 6, dtype=np.int32), (3, 1, 4)).copy()
    q = np.full((3, 1, 4), 0.9, np.float32)       # more than p everywhere (no distribution, but allowed)
    token = np.full((3, 1), 2, np.int32)
    u = np.array([[0.99, 0.05], [0.99, 0.5], [0.99, 0.95]], np.float32)
    out, count = run(x, token, ids, q, u, None, {})
    assert count.tolist() == [1, 1, 1]
    w, _ = weights(x[0, 0].double().numpy())
    c = np.cumsum(w) / w.sum()
    assert out[:, 0].tolist() == [int(np.searchsorted(c, v, side="right")) for v in (0.05, 0.5, 0.95)]


@pytest.mark.parametrize("s", [0, 1, 65, 255])
def test_lengths_of_a_draft(s):
    """None at all, one, more than a wave looks at, the longest."""
    rng = np.random.default_rng(s)
    n = 90
    x = values("noise", 3 * (s + 1), n, "fp32", rng).view(3, s + 1, n)
    token, ids, q = drafts(x, 8, rng) if s else (np.zeros((3, 0), np.int32), np.zeros((3, 0, 8), np.int32),
                                                  np.zeros((3, 0, 8), np.float32))
    u = rng.random((3, s + 1)).astype(np.float32)
    u[1, :s] = 0.0          # accepts whatever has a chance
    got = run(x, token, ids, q, u, None, {})
    assert check(x, token, ids, q, u, None, got, {}) <= 1
    if s:
        assert got[1][1] == s + 1


def test_the_target_s_distribution_comes_out():
    """The point of it: for a grid of u, the first token is distributed as the target's own, whatever the drafter says."""
    n, m = 6, 200
    p_log = torch.tensor([0.3, 1.2, -0.5, 0.9, -2.0, 0.1])
    q = np.array([0.5, 0.05, 0.05, 0.1, 0.2, 0.1], np.float32)
    grid = (np.arange(m) + 0.5) / m
    u = np.stack(np.meshgrid(grid, grid, indexing="ij"), -1).reshape(-1, 2).astype(np.float32)
    p = torch.softmax(p_log.double() / 0.8, 0).numpy()
    seen = np.zeros(n)
    for t in range(n):
        B = len(u)
        x = p_log.expand(B, 2, n).contiguous()
        ids = np.broadcast_to(np.arange(n, dtype=np.int32), (B, 1, n)).copy()
        out, _ = run(x, np.full((B, 1), t, np.int32), ids, np.broadcast_to(q, (B, 1, n)).copy(), u, None,
                     dict(temperature=0.8))
        seen += q[t] * np.bincount(out[:, 0].cpu().numpy(), minlength=n) / B
    # each share is a sum over two grids of m points: off by 1 / m for either at most
    assert np.abs(seen - p).max() <= 2.0 / m


def test_rows_of_a_wider_tensor_another_stream_and_replays():
    rng = np.random.default_rng(15)
    B, s, n = 4, 3, 5003
    wide = values("model", B * (s + 1), n + 5, "bf16", rng).view(B, s + 1, n + 5)
    x = wide[:, :, 1:n + 1]
    token, ids, q = drafts(x, 16, rng)
    u = rng.random((B, s + 1)).astype(np.float32)
    on = lambda t: torch.from_numpy(t).to(DEV)  # noqa: E731
    d_wide, d_u = wide.to(DEV), on(u)
    args = dict(idx=on(ids), probs=on(q), temperature=0.9, top_p=0.9)
    d_token = on(token)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = lr.verify(d_wide[:, :, 1:n + 1], d_token, d_u, **args)
    side.synchronize()
    how = dict(T=0.9, p=0.9)
    check(x, token, ids, q, u, None, got, how)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lr.verify(d_wide[:, :, 1:n + 1], d_token, d_u, **args)
    for _ in range(4):
        u = rng.random((B, s + 1)).astype(np.float32)
        d_u.copy_(on(u))
        graph.replay()
        lr.verify(d_wide[:, :, 1:n + 1], d_token, d_u)
        torch.cuda.synchronize()
        check(x, token, ids, q, u, None, out, how)


def test_a_drafter_s_loop():
    """Draft, sample, embed and verify as a speculative decoder calls them, against the same steps in 64 bits."""
    rng = np.random.default_rng(16)
    V, d, r, k, B, s = 4000, 256, 64, 16, 5, 4
    f = lambda *shape, c=1.0: torch.from_numpy((c * rng.standard_normal(shape)).astype(np.float32))  # noqa: E731
    W, E = f(V, d, c=0.4).to(DEV), f(V, d).to(DEV)
    Q = f(r, d, c=d ** -0.5).to(DEV)
    P = (W @ torch.linalg.pinv(Q)).contiguous()          # a head of its own, near the full one
    head = lr.Head(Q, P, W, B_max=B, k_max=k)
    h = f(B, d, c=0.5).to(DEV)
    hs, tokens, ids, probs, us = [h], [], [], [], []
    for _ in range(s):
        idx, _, logits = head.draft(h, k, want_score=False)
        u = torch.from_numpy(rng.random(B).astype(np.float32)).to(DEV)
        token, prob, q = lr.sample(logits, u, idx=idx, temperature=0.9, want_probs=True)
        lists = idx.cpu().numpy()
        for b in range(B):
            w, near = weights(logits[b].cpu().double().numpy(), T=0.9)
            c = np.cumsum(w) / w.sum()
            j = int(np.searchsorted(c, float(u[b]), side="right"))
            assert token[b] == lists[b, j] and abs(float(prob[b]) - w[j] / w.sum()) < 1e-6
        h = 0.5 * h + lr.embed(E, token, scale=0.1)
        assert torch.equal(h, 0.5 * hs[-1] + E[token.long()] * 0.1)
        hs.append(h)
        tokens.append(token)
        ids.append(idx)
        probs.append(q)
    x = torch.stack([head.dense_logits(v) for v in hs], 1)
    u = rng.random((B, s + 1)).astype(np.float32)
    got = lr.verify(x, torch.stack(tokens, 1), torch.from_numpy(u).to(DEV), idx=torch.stack(ids, 1),
                    probs=torch.stack(probs, 1), temperature=0.9, top_k=200, top_p=0.95)
    out = [torch.stack(t, 1).cpu().numpy() for t in (tokens, ids, probs)]
    assert check(x.cpu(), *out, u, None, got, dict(T=0.9, k=200, p=0.95)) == 0
    after = lr.embed(E, got[0])                           # empty slots give rows of zeros
    assert after.shape == (B, s + 1, d) and after[got[0] < 0].abs().sum() == 0
    head.close()


@pytest.mark.parametrize("n,dtype", [(700, "fp32"), (9001, "bf16"), (20001, "fp32")])
def test_large_batches_give_what_small_ones_do(n, dtype):
    """More rows than compute units, under every setting, against the same sequences a few at a time."""
    rng = np.random.default_rng(43)
    names = list(SETTINGS)
    B, s, each = 5 * len(names), 4, 20
    x = values("model", B * (s + 1), n, dtype, rng).view(B, s + 1, n)
    token, ids, q = drafts(x, 16, rng)
    u = rng.random((B, s + 1)).astype(np.float32)
    length = rng.integers(0, s + 1, B).astype(np.int32)
    how = [SETTINGS[names[b % len(names)]] for b in range(B)]
    col = lambda key, other, dt: torch.tensor([h.get(key, other) for h in how], dtype=dt, device=DEV)  # noqa: E731
    f = torch.float32
    args = dict(temperature=col("T", 1.0, f), top_k=col("k", 0, torch.int32), top_p=col("p", 1.0, f),
                min_p=col("m", 0.0, f))
    got = run(x, token, ids, q, u, length, args)
    for b0 in range(0, B, each):
        b = slice(b0, b0 + each)
        part = run(x[b], token[b].copy(), ids[b].copy(), q[b].copy(), u[b].copy(), length[b].copy(),
                   {k: v[b].clone() for k, v in args.items()})
        assert torch.equal(got[0][b], part[0]) and torch.equal(got[1][b], part[1])
    first = slice(0, len(names))
    assert check(x[first], token[first], ids[first], q[first], u[first], length[first], [t[first] for t in got],
                 how[first]) <= 2
