"""The embedding lookup and its gradient against plain implementations in 64 bits."""
import numpy as np
import pytest
import torch

import rank_lm_head_amd as lr

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def tokens(kind, N, V, rng):
    if kind == "zipf":
        t = np.floor(V ** rng.random(N)).astype(np.int64) - 1
        return np.clip(t, 0, V - 1).astype(np.int32)
    if kind == "even":
        return rng.integers(0, V, N).astype(np.int32)
    if kind == "one":
        return np.full(N, V // 2, np.int32)
    if kind == "two":
        return np.where(rng.random(N) < 0.5, 0, V - 1).astype(np.int32)
    t = rng.integers(0, V, N).astype(np.int32)     # some
    t[rng.random(N) < 0.4] = -1
    t[rng.random(N) < 0.1] = min(V, 2 ** 31 - 1)
    t[rng.random(N) < 0.1] = -2 ** 31
    return t


@pytest.mark.parametrize("N,V,d", [(1, 1, 1), (1, 100, 8), (5, 100, 7), (64, 1000, 512), (33, 999, 2049), (300, 50, 5120),
                                   (1000, 4096, 96), (70, 10, 65536), (17, 31, 2048), (3, 5, 2047)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1.0, 71.5, -0.3, 0.0])
def test_lookup(N, V, d, dtype, scale):
    rng = np.random.default_rng(N + d)
    W = torch.from_numpy(rng.standard_normal((V, d)).astype(np.float32)).to(DT[dtype])
    t = tokens("some", N, V, rng)
    out = lr.embed(W.to(DEV), torch.from_numpy(t).to(DEV), scale=scale).cpu().double().numpy()
    want = W.double().numpy()[np.clip(t, 0, V - 1)] * float(np.float32(scale))
    want[(t < 0) | (t >= V)] = 0
    # a product in fp32 (half a step of it), rounded to the type
    assert np.all(np.abs(out - want) <= np.abs(want) * (HALF_STEP[dtype] + 2.0 ** -23))
    if scale == 1.0:
        assert np.array_equal(out, want)


def test_lookup_of_any_shape_and_alignment():
    rng = np.random.default_rng(1)
    big = torch.from_numpy(rng.standard_normal((40, 33)).astype(np.float32)).bfloat16().to(DEV)
    W = big[1:]                                   # rows at odd elements
    t = torch.from_numpy(rng.integers(0, 39, (2, 3, 5)).astype(np.int32)).to(DEV)
    assert torch.equal(lr.embed(W, t), W[t.long()])
    assert lr.embed(W, t[:0]).shape == (0, 3, 5, 33)
    assert torch.equal(lr.embed(W, t[0, 0, 0]), W[t[0, 0, 0].long()])


def test_lookup_keeps_infinities_and_zeroes_missing_rows():
    W = torch.tensor([[float("inf"), float("nan"), 1.0], [2.0, -float("inf"), 3e38]], device=DEV)
    out = lr.embed(W, torch.tensor([1, -1, 0], dtype=torch.int32, device=DEV), scale=2.0)
    assert torch.equal(out[1], torch.zeros(3, device=DEV))
    assert out[0].tolist() == [4.0, -float("inf"), float("inf")] and out[2][0] == float("inf") and out[2][1].isnan()


def test_lookup_past_32_bits():
    """Rows that begin more than 2^32 bytes, and 2^31 elements, into the matrix."""
    V, d = 2 ** 17 + 3, 2 ** 14 + 8
    W = torch.zeros(V, d, dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([0, 65535, 131071, V - 1], dtype=torch.int32, device=DEV)
    for i, r in enumerate(rows.tolist()):
        W[r] = i + 1
    out = lr.embed(W, rows)
    assert torch.equal(out.float(), torch.arange(1.0, 5.0, device=DEV)[:, None].expand(4, d))
    dW = lr.embed_grad(out, rows, V, out=W)
    assert dW.data_ptr() == W.data_ptr()
    assert torch.equal(W[rows.long()].float(), 2 * torch.arange(1.0, 5.0, device=DEV)[:, None].expand(4, d))
    del W
    dW = lr.embed_grad(out, rows, V)
    assert torch.equal(dW[rows.long()], out)
    dW[rows.long()] = 0
    assert not dW.any()


def grad_ref(dY, t, V, scale, old=None):
    """(gradient in 64 bits, sum of the magnitudes that went into it, number of terms)"""
    g = np.zeros((V, dY.shape[1]))
    mag = np.zeros_like(g)
    terms = np.zeros(V)
    live = (t >= 0) & (t < V)
    y = dY.double().numpy()[live]
    np.add.at(g, t[live], y)
    np.add.at(mag, t[live], np.abs(y))
    np.add.at(terms, t[live], 1)
    s = float(np.float32(scale))
    g, mag = g * s, mag * abs(s)
    if old is not None:
        g, mag = g + old.double().numpy(), mag + np.abs(old.double().numpy())
    return g, mag, terms


def check_grad(got, dY, t, V, scale, dtype, old=None):
    g, mag, terms = grad_ref(dY, t, V, scale, old)
    got = got.cpu().double().numpy()
    # terms - 1 additions, one product, and one addition to what was there, each off by half a step of a partial sum, which
    # is at most mag; one rounding to the type
    bound = (terms[:, None] + 2) * 2.0 ** -24 * mag + HALF_STEP[dtype] * (np.abs(g) + (terms[:, None] + 2) * 2.0 ** -24 * mag)
    assert np.all(np.abs(got - g) <= bound)
    none = terms == 0
    assert np.array_equal(got[none], np.zeros_like(g[none]) if old is None else old.double().numpy()[none])


@pytest.mark.parametrize("N,V,d", [(1, 1, 1), (1, 50, 8), (2, 3, 7), (16, 100, 64), (17, 100, 513), (333, 4096, 256),
                                   (1000, 20, 33), (4096, 999, 40), (1023, 511, 520), (5000, 512, 16),
                                   (16384, 3000, 24), (2048, 70000, 16), (512, 5000, 12), (513, 5000, 12), (511, 9001, 3)])
@pytest.mark.parametrize("kind", ["zipf", "even", "one", "two", "some"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient(N, V, d, kind, dtype):
    rng = np.random.default_rng(N + V)
    dY = torch.from_numpy(rng.standard_normal((N, d)).astype(np.float32)).to(DT[dtype])
    t = tokens(kind, N, V, rng)
    for scale, add in ((1.0, False), (-2.5, False), (0.7, True)):
        print(f"[run] {N}x{d} V={V} {kind} {dtype} scale {scale} add {add}", flush=True)
        old = torch.from_numpy(rng.standard_normal((V, d)).astype(np.float32)).to(DT[dtype]) if add else None
        got = lr.embed_grad(dY.to(DEV), torch.from_numpy(t).to(DEV), V, scale=scale,
                            out=old.to(DEV) if add else None)
        check_grad(got, dY, t, V, scale, dtype, old)


@pytest.mark.parametrize("N,V,d", [(16385, 700, 16), (40000, 151936, 16), (70001, 2 ** 20 + 1, 8), (131072, 9, 24),
                                   (300, 2 ** 27 - 5, 1), (90, 2 ** 24, 2), (90, 2 ** 24 + 1, 2), (3000, 2 ** 20 - 3, 4), (16384, 2 ** 18 + 1, 8), (600001, 30000, 8)])
@pytest.mark.parametrize("kind", ["zipf", "some"])
def test_gradient_of_many_rows(N, V, d, kind):
    """The sort over several blocks: more places than one block sorts, or tokens and places past one word."""
    rng = np.random.default_rng(N)
    dY = torch.from_numpy(rng.standard_normal((N, d)).astype(np.float32))
    t = tokens(kind, N, V, rng)
    got = lr.embed_grad(dY.to(DEV), torch.from_numpy(t).to(DEV), V)
    live = (t >= 0) & (t < V)
    rows = np.unique(t[live])
    small = np.searchsorted(rows, t[live]).astype(np.int32)
    check_grad(got[torch.from_numpy(rows.astype(np.int64)).to(DEV)], dY[torch.from_numpy(live)], small, len(rows), 1.0, "fp32")
    got[torch.from_numpy(rows.astype(np.int64)).to(DEV)] = 0
    assert not got.any()


def test_gradient_does_not_vary():
    rng = np.random.default_rng(3)
    for N in (5000, 50000):
        dY = torch.from_numpy(rng.standard_normal((N, 72)).astype(np.float32)).to(DEV)
        t = torch.from_numpy(tokens("zipf", N, 5000, rng)).to(DEV)
        a = lr.embed_grad(dY, t, 5000)
        lr.embed_grad(dY.flip(0).contiguous(), t, 5000)
        assert torch.equal(a, lr.embed_grad(dY, t, 5000))


def test_gradient_at_any_alignment_and_without_rows():
    rng = np.random.default_rng(4)
    flat = torch.from_numpy(rng.standard_normal(1 + 50 * 33).astype(np.float32)).bfloat16()
    t = tokens("some", 50, 20, rng)
    dY = flat.to(DEV)[1:].view(50, 33)
    room = torch.zeros(1 + 20 * 33, dtype=torch.bfloat16, device=DEV)
    got = lr.embed_grad(dY, torch.from_numpy(t).to(DEV), 20, out=room[1:].view(20, 33))
    check_grad(got, flat[1:].view(50, 33), t, 20, 1.0, "bf16")
    assert room[0] == 0
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    assert not lr.embed_grad(torch.zeros(0, 5, device=DEV), none, 7).any()
    old = torch.ones(7, 5, device=DEV)
    assert torch.equal(lr.embed_grad(torch.zeros(0, 5, device=DEV), none, 7, out=old), torch.ones(7, 5, device=DEV))


def test_gradient_leaves_other_rows_as_they_were():
    """With `out`, rows of tokens that do not occur keep every bit, NaN among them."""
    old = torch.full((9, 12), float("nan"), device=DEV)
    old[4] = 1.0
    t = torch.tensor([4, 4, -1, 9], dtype=torch.int32, device=DEV)
    got = lr.embed_grad(torch.ones(4, 12, device=DEV), t, 9, scale=0.5, out=old)
    assert (got[4] == 2.0).all() and got.isnan().sum() == 8 * 12


def test_rows_of_missing_tokens_are_not_read():
    dY = torch.ones(6, 40, device=DEV)
    dY[2], dY[5] = float("nan"), float("inf")
    t = torch.tensor([1, 1, -1, 0, 1, 99], dtype=torch.int32, device=DEV)
    got = lr.embed_grad(dY, t, 3)
    assert got.isfinite().all() and got[1, 0] == 3 and got[0, 0] == 1


def test_capture_and_another_stream():
    rng = np.random.default_rng(5)
    for N, V in ((700, 300), (20000, 300)):
        dY = torch.from_numpy(rng.standard_normal((N, 48)).astype(np.float32)).to(DEV)
        t = torch.from_numpy(tokens("zipf", N, V, rng)).to(DEV)
        W = torch.from_numpy(rng.standard_normal((V, 48)).astype(np.float32)).to(DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a, b = lr.embed(W, t), lr.embed_grad(dY, t, V)
        side.synchronize()
        assert torch.equal(a, W[t.long()]) and torch.equal(b, lr.embed_grad(dY, t, V))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = lr.embed(W, t, scale=2.0)
            g = lr.embed_grad(dY, t, V, scale=3.0)
        for _ in range(4):
            t.copy_(torch.from_numpy(tokens("even", N, V, rng)))
            dY.normal_()
            graph.replay()
            lr.embed_grad(dY, t, V)
            torch.cuda.synchronize()
            assert torch.equal(y, W[t.long()] * 2.0) and torch.equal(g, lr.embed_grad(dY, t, V, scale=3.0))


def test_autograd():
    """embedding()'s gradient against the formula's and against differences (the function is linear: a step of 1 is exact
    up to roundings)."""
    rng = np.random.default_rng(6)
    V, d, N = 30, 20, 90
    W = torch.from_numpy(rng.standard_normal((V, d)).astype(np.float32)).to(DEV).requires_grad_()
    t = torch.from_numpy(tokens("some", N, V, rng)).to(DEV).view(9, 10)
    c = torch.from_numpy(rng.standard_normal((9, 10, d)).astype(np.float32)).to(DEV)
    (lr.embedding(W, t, scale=1.5) * c).sum().backward()
    check_grad(W.grad, c.view(N, d).cpu(), t.view(N).cpu().numpy(), V, 1.5, "fp32")
    f = lambda w: (lr.embed(w, t, scale=1.5).double() * c.double()).sum()  # noqa: E731
    for v, j in ((0, 0), (7, 3), (29, 19)):
        step = torch.zeros_like(W)
        step[v, j] = 1.0
        diff = float(f(W.detach() + step) - f(W.detach() - step)) / 2
        assert abs(diff - float(W.grad[v, j])) <= 1e-4
    W.grad = None
    lr.embedding(W, t).sum().backward()            # the gradient that arrives is one number, expanded
    live = t[(t >= 0) & (t < V)].long()
    assert torch.equal(W.grad[:, 0], torch.bincount(live, minlength=V).float())
    assert not lr.embedding(W.detach(), t).requires_grad
    with torch.no_grad():
        assert not lr.embedding(W, t).requires_grad


def test_autograd_refuses_capture():
    W = torch.zeros(5, 8, device=DEV, requires_grad=True)
    t = torch.zeros(3, dtype=torch.int32, device=DEV)
    lr.embedding(W, t).sum().backward()
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(graph):
            lr.embedding(W, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad():   # without gradients it can
        with torch.cuda.graph(graph):
            y = lr.embedding(W, t)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, torch.zeros(3, 8, device=DEV))


@pytest.mark.parametrize("N", [3, 300, 900, 17000])
def test_gradient_past_32_bits(N):
    """A matrix of 2.9e9 elements, 5.7 GB, which held other values."""
    V, d = 72000, 40000
    rng = np.random.default_rng(N)
    dY = torch.from_numpy(rng.standard_normal((min(N, 64), d)).astype(np.float32)).bfloat16().to(DEV)
    dY = dY.repeat(-(-N // len(dY)), 1)[:N].contiguous()
    t = rng.choice(V, N, replace=False).astype(np.int32)
    t[0] = V - 1 if V - 1 not in t else t[0]
    torch.full((V, d), 7.0, dtype=torch.bfloat16, device=DEV)      # freed: the result may take its place
    dW = lr.embed_grad(dY, torch.from_numpy(t).to(DEV), V)
    at = torch.from_numpy(t).long().to(DEV)
    for i in range(0, N, 2000):
        assert torch.equal(dW[at[i:i + 2000]], dY[i:i + 2000])     # one row a token: the row itself
        dW[at[i:i + 2000]] = 0
    for v in range(0, V, 8000):
        assert not dW[v:v + 8000].any()
