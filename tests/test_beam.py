"""Beam selection and state reordering against the definition in 64 bits."""
import ctypes

import numpy as np
import pytest
import torch

import gen
import rank_lm_head_amd as lr
from parity_util import dev
from rank_lm_head_amd import _lib

DEV = "cuda:0"
A = ctypes.c_void_p(0x10000)        # aligned stand-ins: never dereferenced
MIS = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10002)
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
NEG = float("-inf")


# ------------------------------------------------------------------ refusals

def _select(dtype=_lib.FP32, x=A, ld=100, idx=None, score=A, ended=None, B=2, m=3, n=100, nb=4, o=A, ob=A, ot=A, ws=A,
            nbytes=1 << 40):
    return _lib.load().lrhead_beam_select(dtype, x, ld, idx, score, ended, 0, B, m, n, nb, o, ob, ot, ws, nbytes, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=2), _lib.EDTYPE), (dict(m=0), _lib.ERANGE), (dict(m=65), _lib.ERANGE), (dict(nb=0), _lib.ERANGE),
    (dict(nb=65), _lib.ERANGE), (dict(n=0), _lib.ERANGE), (dict(n=1 << 31, ld=1 << 31), _lib.ERANGE),
    (dict(B=-1), _lib.ERANGE), (dict(B=1 << 20, m=64, n=1 << 30, ld=1 << 30), _lib.ERANGE), (dict(ld=99), _lib.ERANGE),
    (dict(x=None), _lib.EINVAL), (dict(score=None), _lib.EINVAL), (dict(o=None), _lib.EINVAL),
    (dict(ot=None), _lib.EINVAL), (dict(ws=None), _lib.EINVAL), (dict(x=ODD), _lib.EALIGN),
    (dict(idx=ODD), _lib.EALIGN), (dict(score=ODD), _lib.EALIGN), (dict(ws=MIS), _lib.EALIGN),
    (dict(B=1 << 20, m=17, n=65), _lib.ERANGE), (dict(ob=MIS), _lib.EALIGN), (dict(nbytes=16), _lib.EWORKSPACE),
])
def test_select_refuses_bad_arguments_before_hip(kwargs, code):
    assert _select(**kwargs) == code
    assert _lib.load().lrhead_last_error()


def test_select_of_nothing():
    assert _select(B=0, x=None, o=None) == _lib.OK


def _states(*rows):
    arr = (_lib.State * len(rows))()
    for s, (src, dst, segs, positions, nbytes) in zip(arr, rows):
        s.src, s.dst, s.segs, s.positions, s.position_bytes = src, dst, segs, positions, nbytes
    return arr


@pytest.mark.parametrize("rows,code", [
    ([(0x10000, 0x10010, 1, 1, 16)], _lib.EINVAL),                                 # dst inside src (2 x 2 x 16 bytes)
    ([(0x10000, 0x20000, 1, 1, 16), (0x30000, 0x20010, 1, 1, 16)], _lib.EINVAL),   # two dst
    ([(0x10000, 0x20000, 1, 1, 16), (0x20030, 0x40000, 1, 1, 16)], _lib.EINVAL),   # a dst and another src
    ([(0x10000, 0x10000, 1, 1, 16)], _lib.EINVAL),
    ([(None, 0x20000, 1, 1, 16)], _lib.EINVAL),
    ([(0x10000, 0x20000, -1, 1, 16)], _lib.ERANGE),
    ([(0x10000, 0x20000, 1 << 40, 1 << 40, 16)], _lib.ERANGE),
])
def test_reorder_refuses_bad_states_before_hip(rows, code):
    arr = _states(*rows)
    assert _lib.load().lrhead_reorder(arr, len(arr), A, None, 2, 2, 2, None) == code


def test_reorder_refuses_bad_sizes_and_accepts_nothing():
    lib = _lib.load()
    arr = _states((0x10000, 0x20000, 1, 1, 16))
    assert lib.lrhead_reorder(arr, 1, A, None, -1, 2, 2, None) == _lib.ERANGE
    assert lib.lrhead_reorder(arr, 1, A, None, 1, 0, 2, None) == _lib.ERANGE
    assert lib.lrhead_reorder(arr, -1, A, None, 1, 2, 2, None) == _lib.ERANGE
    assert lib.lrhead_reorder(arr, 1025, A, None, 1, 2, 2, None) == _lib.ERANGE
    assert lib.lrhead_reorder(arr, 1, None, None, 1, 2, 2, None) == _lib.EINVAL
    assert lib.lrhead_reorder(None, 0, None, None, 1, 2, 2, None) == _lib.OK
    assert lib.lrhead_reorder(arr, 1, None, None, 0, 2, 2, None) == _lib.OK
    empty = _states((None, None, 1, 0, 16))
    assert lib.lrhead_reorder(empty, 1, A, None, 1, 2, 2, None) == _lib.OK


def test_bindings_refuse_cpu_tensors():
    with pytest.raises(ValueError):
        lr.beam_select(torch.zeros(1, 2, 8), torch.zeros(1, 2), 2)
    with pytest.raises(ValueError):
        lr.reorder(torch.zeros(1, 2, 8), torch.zeros(1, 2, dtype=torch.int32))


# ----------------------------------------------------------------- reference

def reference(x, score, nb, idx=None, ended=None, end_id=0):
    """Totals, beams and tokens in candidate order, in 64 bits; and the gap
    from each place to the next one."""
    x = x.detach().cpu().double().numpy()
    score = score.cpu().double().numpy()
    B, m, n = x.shape
    out = np.full((B, nb), -np.inf)
    beam = np.full((B, nb), -1)
    token = np.full((B, nb), -1)
    gap = np.full((B, nb), np.inf)
    for b in range(B):
        tot, bm, col, tok = [], [], [], []
        for i in range(m):
            if ended is not None and bool(ended[b, i]):
                tot.append([score[b, i]]); bm.append([i]); col.append([0]); tok.append([end_id])
                continue
            v = x[b, i].copy()
            v[np.isnan(v)] = -np.inf
            ids = np.arange(n) if idx is None else idx[b, i].cpu().numpy()
            v[ids < 0] = -np.inf
            hi = v.max()
            if hi == -np.inf:
                continue
            with np.errstate(over="ignore", under="ignore"):
                log = np.log(np.exp(v - hi).sum())
            keep = np.argsort(-v, kind="stable")[:nb + 1]
            tot.append(v[keep] - hi - log + score[b, i]); bm.append(np.full(len(keep), i)); col.append(keep); tok.append(ids[keep])
        if not tot:
            continue
        tot, bm, col, tok = (np.concatenate([np.asarray(y) for y in z]) for z in (tot, bm, col, tok))
        good = tot > -np.inf
        tot, bm, col, tok = tot[good], bm[good], col[good], tok[good]
        order = np.lexsort((col, bm, -tot))
        c = min(nb, len(order))
        out[b, :c], beam[b, :c], token[b, :c] = tot[order][:c], bm[order][:c], tok[order][:c]
        t = tot[order]
        gap[b, :min(c, len(t) - 1)] = (t[:-1] - t[1:])[:c]
    return out, beam, token, gap


def check(x, score, nb, idx=None, ended=None, end_id=0):
    got = lr.beam_select(x, score, nb, idx=idx, ended=ended, end_id=end_id)
    torch.cuda.synchronize()
    s, bm, tk = (g.cpu().numpy() for g in got)
    out, beam, token, gap = reference(x, score, nb, idx, ended, end_id)
    with np.errstate(invalid="ignore"):
        err = np.abs(s.astype(np.float64) - out)
    err[np.isneginf(out) & np.isneginf(s)] = 0
    # fp32 output: half a step; the sum of exponentials: a few half steps of fp32 of itself
    assert np.all(err <= 2.0 ** -24 * np.abs(np.where(np.isneginf(out), 0, out)) + 1e-6), err.max()
    # equal totals (of one beam, or of equal beams) have a fixed order; others closer than the sums' error may swap
    near = (gap > 0) & (gap < 2e-6)
    sure = ~(near | np.roll(near, 1, axis=1) & (np.arange(nb) > 0))
    assert np.array_equal(bm[sure], beam[sure]) and np.array_equal(tk[sure], token[sure])
    assert sure.mean() > 0.9
    return got


def draw(B, m, n, dt, seed, lists=False):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, m, n, generator=g) * 2.5
    score = -10 * torch.rand(B, m, generator=g)
    ids = torch.randint(0, 100000, (B, m, n), generator=g, dtype=torch.int32).to(DEV) if lists else None
    return x.to(DT[dt]).to(DEV), score.to(DEV), ids


# ----------------------------------------------------------------- on the GPU

@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("B,m,n,nb", [
    (1, 1, 1, 1),
    (2, 3, 1, 5),           # more slots than candidates
    (1, 1, 5, 64),
    (3, 4, 63, 4), (3, 4, 64, 8), (3, 4, 65, 8),     # either side of the one-launch form
    (5, 64, 64, 64),        # the most beams and slots
    (2, 64, 200, 64),
    (1, 2, 1023, 3), (1, 2, 1024, 3), (2, 1, 1025, 33),
    (7, 5, 32003, 10),      # rows that start off 16 bytes
    (1, 4, 151936, 4),
    (1, 1, 300007, 64),
    (40, 8, 20001, 17),     # longer slices
    (300, 4, 9000, 2),      # the longest
])
def test_select(B, m, n, nb, dt):
    x, score, _ = draw(B, m, n, dt, seed=B * 31 + n)
    check(x, score, nb)


@pytest.mark.gpu
@pytest.mark.parametrize("B,m,n,nb", [(64, 8, 32, 8), (3, 5, 64, 64), (2, 3, 500, 9)])
def test_select_over_candidate_lists(B, m, n, nb):
    x, score, ids = draw(B, m, n, "fp32", seed=n, lists=True)
    ids[0, 0, ::3] = -1              # empty slots by id
    x[1, 1, 5:] = float("nan")       # and by logit
    ids[1, 0] = -1                   # a beam with none
    check(x, score, nb, idx=ids)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [40, 5000])
def test_masks_and_ends(n, dt):
    B, m, nb = 6, 4, 6
    x, score, _ = draw(B, m, n, dt, seed=n + 1)
    low = torch.finfo(DT[dt]).min
    x[0, 1] = NEG                    # a beam without a token
    x[1] = NEG                       # a sequence without one
    x[2, 0] = low                    # all at the type's lowest value: equal, not forbidden
    x[2, 1, : n // 2] = low
    x[3, 2, 3:] = NEG                # three tokens left
    x[3, 3] = float("nan")
    score[4, 1:] = NEG               # the first step: one beam
    score[5, 2] = float("nan")
    ended = torch.zeros(B, m, dtype=torch.bool, device=DEV)
    ended[0, 0] = ended[0, 1] = ended[3, 3] = True
    ended[4, 1] = True               # ended, but without a score
    check(x, score, nb)
    s, bm, tk = check(x, score, nb, ended=ended, end_id=7)
    assert (tk[0][(bm[0] == 0) | (bm[0] == 1)] == 7).all()
    s1, b1, t1 = lr.beam_select(x[1:2], score[1:2], nb)
    assert torch.isneginf(s1).all() and (b1 == -1).all() and (t1 == -1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["fp32", "bf16"])
@pytest.mark.parametrize("n", [50, 3000, 70000])
def test_ties_go_to_the_lower_beam_then_column(n, dt):
    B, m, nb = 2, 3, 12
    x = torch.zeros(B, m, n, dtype=DT[dt], device=DEV)
    score = torch.zeros(B, m, device=DEV)
    s, bm, tk = lr.beam_select(x, score, nb)
    assert (bm == 0).all() and torch.equal(tk[0].cpu(), torch.arange(nb, dtype=torch.int32))
    x[:, 1, n - 5:] = 1.0            # the best, at the row's end
    x[:, 2, n - 5:] = 1.0
    s, bm, tk = lr.beam_select(x, score, nb)
    want = [1] * 5 + [2] * 5
    assert bm[1, :10].tolist() == want and tk[1, :5].tolist() == list(range(n - 5, n))
    assert tk[1, 5:10].tolist() == list(range(n - 5, n)) and bm[1, 10:].tolist() == [0, 0]
    x[:, 0, 3] = -0.0                # -0 and +0 are the same logit
    s, bm, tk = lr.beam_select(x[:, :1].contiguous(), score[:, :1].contiguous(), 5)
    assert tk[0].tolist() == [0, 1, 2, 3, 4]


@pytest.mark.gpu
def test_best_in_one_thread_and_ascending_rows():
    """The nb best side by side in one 16-byte chunk, and a row in ascending order."""
    x, score, _ = draw(2, 2, 50000, "bf16", seed=2)
    x[0, 0, 4096:4104] = torch.arange(20, 28, device=DEV).bfloat16()
    check(x, score, 8)
    y = torch.linspace(-5, 5, 50000, device=DEV).repeat(1, 2, 1).contiguous()
    check(y, score[:1].contiguous(), 64)


@pytest.mark.gpu
def test_rows_of_a_wider_matrix():
    x, score, _ = draw(3, 4, 2100, "fp32", seed=4)
    want = lr.beam_select(x[:, :, :2000].contiguous(), score, 5)
    got = lr.beam_select(x[:, :, :2000], score, 5)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = lr.beam_select(x[:, :, 1:2001], score, 5)     # rows off 16 bytes
    want = lr.beam_select(x[:, :, 1:2001].contiguous(), score, 5)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = lr.beam_select(x[:, ::2], score[:, ::2].contiguous(), 5)   # every second row: evenly spaced as well
    want = lr.beam_select(x[:, ::2].contiguous(), score[:, ::2].contiguous(), 5)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for bad in (x[:, 1:3], x[:, :, ::2], x[:, :1].expand(3, 4, 2100)):
        with pytest.raises(ValueError):
            lr.beam_select(bad, score[:, :bad.shape[1]].contiguous(), 5)


@pytest.mark.gpu
@pytest.mark.parametrize("n,nb", [(262144 + 900, 64), (600001, 7), (1100000, 33)])
def test_many_slices(n, nb):
    """One long row or two: more slices than a wave's lanes hold at once."""
    x, score, _ = draw(1, 2, n, "fp32", seed=n)
    check(x, score, nb)
    check(x[:, :1].contiguous(), score[:, :1].contiguous(), nb)
    up = torch.linspace(-9, 9, n, device=DEV).repeat(1, 2, 1).contiguous()   # all of the best in the last slice
    check(up, score, nb)


@pytest.mark.gpu
def test_inputs_off_16_bytes():
    x, score, _ = draw(5, 3, 900, "bf16", seed=9)
    ids = torch.randint(0, 5000, (5, 3, 900), dtype=torch.int32, device=DEV)
    ended = torch.rand(5, 3, device=DEV) < 0.3
    got = lr.beam_select(x[1:], score[1:], 4, idx=ids[1:], ended=ended[1:], end_id=2)
    want = lr.beam_select(x[1:].clone(), score[1:].clone(), 4, idx=ids[1:].clone(), ended=ended[1:].clone(), end_id=2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows that start behind 2^32 bytes."""
    n = 151936
    big = torch.full((1, 64, n * 120), -30.0, dtype=torch.float32, device=DEV)   # 4.7 GB
    big[0, 63, n * 120 - 1] = 5.0
    big[0, 62, 7] = 5.0
    s, bm, tk = lr.beam_select(big, torch.zeros(1, 64, device=DEV), 2)
    assert bm.tolist() == [[62, 63]] and tk.tolist() == [[7, n * 120 - 1]]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int8, torch.float64, torch.bool])
@pytest.mark.parametrize("shape", [(1, 1, 8), (3, 4, 5120), (2, 5, 7), (4, 3, 2, 9, 3), (2, 2, 3, 4097)])
def test_reorder_whole_states(shape, dtype):
    g = torch.Generator().manual_seed(1)
    x = torch.randint(0, 2 if dtype == torch.bool else 100, shape, generator=g).to(dtype).to(DEV)
    B, m = shape[:2]
    parent = torch.randint(0, m, (B, m + 2), generator=g, dtype=torch.int32).to(DEV)
    got = lr.reorder(x, parent)
    want = x[torch.arange(B, device=DEV)[:, None], parent.long()]
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_reorder_keeps_what_is_not_moved():
    B, m, nb, heads, T, w = 5, 3, 4, 2, 33, 8
    g = torch.Generator().manual_seed(2)
    xs = [torch.randn(B, m, heads, T, w, generator=g).to(DEV), torch.randn(B, m, heads, T, w, generator=g).bfloat16().to(DEV)]
    parent = torch.randint(0, m, (B, nb), generator=g, dtype=torch.int32).to(DEV)
    parent[1, 2] = -1
    parent[2, 0] = m
    parent[3, 3] = 2 ** 31 - 1
    length = torch.tensor([0, 1, 33, 40, -3], dtype=torch.int32, device=DEV)
    outs = [torch.full((B, nb, heads, T, w), 9.0, dtype=x.dtype, device=DEV) for x in xs]
    got = lr.reorder(xs, parent, length=length, out=outs)
    assert all(a is b for a, b in zip(got, outs))
    fresh = lr.reorder(xs, parent, length=length)
    for x, o, f in zip(xs, outs, fresh):
        want = torch.full_like(o, 9.0)
        for b in range(B):
            n = min(max(int(length[b]), 0), T)
            for j in range(nb):
                p = int(parent[b, j])
                if 0 <= p < m:
                    want[b, j, :, :n] = x[b, p, :, :n]
        assert torch.equal(o, want)
        assert torch.equal(f, torch.where(want == 9.0, torch.zeros_like(want), want))


@pytest.mark.gpu
def test_reorder_positions_along_other_dimensions():
    x = torch.arange(2 * 3 * 5 * 4, dtype=torch.float32, device=DEV).view(2, 3, 5, 4)
    parent = torch.tensor([[2, 0], [1, 1]], dtype=torch.int32, device=DEV)
    length = torch.tensor([2, 3], dtype=torch.int32, device=DEV)
    for dim in (2, 3, -1):
        got = lr.reorder(x, parent, length=length, dim=dim)
        want = torch.zeros(2, 2, 5, 4, device=DEV)
        for b in range(2):
            for j in range(2):
                s = x[b, int(parent[b, j])]
                n = int(length[b])
                if dim == 2:
                    want[b, j, :n] = s[:n]
                else:
                    want[b, j, :, :n] = s[:, :n]
        assert torch.equal(got, want)
    with pytest.raises(ValueError):
        lr.reorder(x, parent, length=length, dim=1)


@pytest.mark.gpu
def test_reorder_many_states_and_odd_addresses():
    B, m, nb = 2, 3, 3
    g = torch.Generator().manual_seed(3)
    parent = torch.randint(0, m, (B, nb), generator=g, dtype=torch.int32).to(DEV)
    xs = [torch.randn(B, m, 5 + i, generator=g).to(DEV) for i in range(70)]     # several launches
    xs.append(torch.zeros(B, m, 0, device=DEV))                                 # nothing in it
    raw = torch.arange(1 + B * m * 11, dtype=torch.uint8, device=DEV)
    xs.append(raw[1:].view(B, m, 11))                                           # off by one byte
    got = lr.reorder(xs, parent)
    for x, o in zip(xs, got):
        assert torch.equal(o, x[torch.arange(B, device=DEV)[:, None], parent.long()])
    with pytest.raises(lr.LrheadError):
        lr.reorder(xs[0], parent, out=xs[0])
    assert lr.reorder([], parent) == []


@pytest.mark.gpu
def test_reorder_of_many_short_segments():
    """More blocks than one row of a launch."""
    g = torch.Generator().manual_seed(5)
    x = torch.randint(0, 100, (1, 2, 600001, 3), generator=g, dtype=torch.uint8).to(DEV)
    got = lr.reorder(x, torch.tensor([[1, 0]], dtype=torch.int32, device=DEV),
                     length=torch.tensor([2], dtype=torch.int32, device=DEV), dim=-1)
    want = x[:, [1, 0]].clone()
    want[..., 2] = 0
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_reorder_past_32_bits():
    x = torch.zeros(1, 3, (1 << 31) + 4096, dtype=torch.uint8, device=DEV)   # 6.4 GB
    x[0, 1, -5:] = 3
    x[0, 2, -7:] = 4
    got = lr.reorder(x, torch.tensor([[2, 1]], dtype=torch.int32, device=DEV))
    assert torch.equal(got[0, 0], x[0, 2]) and torch.equal(got[0, 1], x[0, 1])


@pytest.mark.gpu
def test_graph_replays_match_eager_calls():
    B, m, n, nb = 3, 4, 9000, 4
    sets = [draw(B, m, n, "fp32", seed=s)[:2] for s in (1, 2, 3)]
    state = torch.randn(B, m, 64, device=DEV)
    held = [y.clone() for y in sets[0]]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s, bm, tk = lr.beam_select(held[0], held[1], nb)
            moved = lr.reorder(state, bm)
        graphs.append((g, (s, bm, tk, moved)))
    for x, score in sets + sets[:1]:
        held[0].copy_(x)
        held[1].copy_(score)
        for g, _ in graphs:
            g.replay()
        want = lr.beam_select(x, score, nb)
        torch.cuda.synchronize()
        want = (*want, lr.reorder(state, want[1]))
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_side_stream_matches():
    x, score, _ = draw(4, 4, 30000, "bf16", seed=6)
    want = lr.beam_select(x, score, 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = lr.beam_select(x, score, 6)
        moved = lr.reorder(x, got[1])
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(moved, x[torch.arange(4, device=DEV)[:, None], want[1].long()])


@pytest.mark.gpu
def test_beams_over_the_draft_head():
    """The operators as they are used: each step drafts every beam's
    candidates, selects over all of them and moves the beams' rows."""
    V, d, r, B, m, k = 2000, 128, 32, 3, 4, 8
    inp = gen.make_custom(V, d, r, B * m, "bf16", seed=5)
    t = {x: dev(inp[x], DEV) for x in ("Q", "P", "W", "H")}
    head = lr.Head(t["Q"], t["P"], t["W"], B_max=B * m, k_max=k)
    H = t["H"].clone()
    score = torch.zeros(B, m, device=DEV)
    score[:, 1:] = NEG               # all beams start from one
    ended = torch.zeros(B, m, dtype=torch.bool, device=DEV)
    for step in range(4):
        idx, _, logits = head.draft(H, k)
        ids, lg = idx.view(B, m, k), logits.view(B, m, k)
        new, beam, token = check(lg, score, m, idx=ids, ended=ended, end_id=1)
        H = lr.reorder(H.view(B, m, d), beam)
        H = (H.float() + 0.3 * t["W"][token.long()].float()).bfloat16().view(B * m, d)
        ended = ended.gather(1, beam.long()) | (token % 5 == 0)
        score = new
    assert bool((score[:, 1:] <= score[:, :-1]).all())
    head.close()
