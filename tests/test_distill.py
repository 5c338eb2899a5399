"""Distillation from a teacher's top logits against the definition in 64 bits.

Tolerances count roundings. A score is off by at most r half steps of fp32 of
the sum of its products' magnitudes; q by that (relatively), by the roundings
of the exponent and by two steps of the exponential; in bf16 the weights of
the gradients' sums and the gradients themselves are rounded once more each.
"""
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
H32 = torch.finfo(torch.float32).eps / 2   # half a step of fp32


# ------------------------------------------------------------------ refusals

def _distill(dtype=_lib.BF16, V=1000, r=16, P=A, Z=A, N=4, idx=A, lg=A, k=4, T=1.0, loss=A, lse=A, grad=A, ws=A,
             n=1 << 40):
    return _lib.load().lrhead_distill(dtype, V, r, P, Z, N, idx, lg, k, T, loss, lse, grad, ws, n, None)


def _grad(dtype=_lib.BF16, V=1000, r=16, P=A, Z=A, N=4, idx=A, lg=A, k=4, T=1.0, lse=A, grad=A, w=A, dZ=A, dP=A, ws=A,
          n=1 << 40):
    return _lib.load().lrhead_distill_grad(dtype, V, r, P, Z, N, idx, lg, k, T, lse, grad, w, dZ, dP, ws, n, None)


@pytest.mark.parametrize("call", [_distill, _grad])
@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=2), _lib.EDTYPE), (dict(V=0), _lib.ERANGE), (dict(V=1 << 31), _lib.ERANGE), (dict(r=12), _lib.ERANGE),
    (dict(r=520), _lib.ERANGE), (dict(N=-1), _lib.ERANGE), (dict(N=(1 << 20) + 1), _lib.ERANGE),
    (dict(k=0), _lib.ERANGE), (dict(k=65), _lib.ERANGE), (dict(T=0.0), _lib.ERANGE), (dict(T=-1.0), _lib.ERANGE),
    (dict(T=float("nan")), _lib.ERANGE), (dict(T=float("inf")), _lib.ERANGE), (dict(P=None), _lib.EINVAL),
    (dict(idx=None), _lib.EINVAL), (dict(lse=None), _lib.EINVAL), (dict(ws=None), _lib.EINVAL),
    (dict(Z=MIS), _lib.EALIGN), (dict(grad=MIS), _lib.EALIGN), (dict(idx=ODD), _lib.EALIGN),
    (dict(lse=ODD), _lib.EALIGN), (dict(n=64), _lib.EWORKSPACE),
    (dict(dtype=_lib.FP32, V=1 << 28), _lib.ERANGE), (dict(V=1 << 28, N=1 << 20), _lib.ERANGE),
])
def test_calls_refuse_bad_arguments_before_hip(call, kwargs, code):
    assert call(**kwargs) == code
    assert _lib.load().lrhead_last_error()


def test_gradient_of_z_needs_the_forward_gradient():
    assert _grad(grad=None) == _lib.EINVAL


def test_workspace_sizes():
    ws = _lib.load().lrhead_distill_workspace_bytes
    assert ws(_lib.BF16, 151936, 128, 4096, 32) > 0
    for bad in [(3, 100, 16, 1, 1), (_lib.BF16, 0, 16, 1, 1), (_lib.BF16, 100, 15, 1, 1), (_lib.BF16, 100, 16, -1, 1),
                (_lib.BF16, 100, 16, 1, 65), (_lib.FP32, 1 << 27, 16, 1, 1), (_lib.BF16, 1 << 25, 128, 1 << 20, 1)]:
        assert ws(*bad) == 0


def test_binding_refuses_cpu_and_mismatched_tensors():
    Z, P = torch.zeros(3, 16), torch.zeros(50, 16)
    idx, t = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, 4)
    with pytest.raises(ValueError):
        lr.distill(Z, P, idx, t)
    with pytest.raises(ValueError):
        lr.distill_loss(Z, P, idx, t)
    with pytest.raises(ValueError):
        lr.distill(Z, P.bfloat16(), idx, t)
    with pytest.raises(ValueError):
        lr.distill(Z, P[:, :8], idx, t)


# ----------------------------------------------------------------- reference

def reference(Z, P, idx, t, T, w):
    """loss, lse, dloss/dz, dZ, dP in 64 bits, and the magnitudes that the tolerances need."""
    Z, P, t, w = Z.double().cpu(), P.double().cpu(), t.double().cpu(), w.double().cpu()
    idx = idx.long().cpu()
    V = P.shape[0]
    live = w != 0
    Z = torch.where((live | True)[:, None], Z, 0.0)
    real = (idx >= 0) & (idx < V) & (t > -torch.inf)
    any_ = real.any(1)
    te = torch.where(real, t / T, -torch.inf)
    te = te - torch.where(any_, te.amax(1), 0.0)[:, None]
    e = torch.exp(te)
    p = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    logp = torch.where(p > 0, torch.log(p), 0.0)
    s = Z @ P.T / T
    lse = torch.logsumexp(s, 1)
    at = s.gather(1, idx.clamp(0, V - 1))
    loss = torch.where(any_, torch.where(p > 0, p * (logp - at + lse[:, None]), 0.0).sum(1), 0.0)
    q = torch.where(any_[:, None], torch.exp(s - lse[:, None]), 0.0)
    pv = torch.zeros_like(q).scatter_add_(1, idx.clamp(0, V - 1), p)
    grad = torch.where(any_[:, None], (q - pv) @ P / T, 0.0)
    c = torch.where(any_ & live, w / T, 0.0)
    safe = torch.where((any_ & live)[:, None], Z, 0.0)
    qs, ps = torch.where(live[:, None], q, 0.0), torch.where(live[:, None], pv, 0.0)
    dP = (c[:, None] * (qs - ps)).T @ safe
    # magnitudes
    ok = torch.isfinite(Z).all(1)
    size = (Z[ok].abs() @ P.abs().T).max().item() / T if ok.any() else 0.0
    top = (s[ok].abs().max().item() + lse[ok].abs().max().item()) if ok.any() else 0.0
    return {"loss": loss, "lse": lse, "grad": grad, "dZ": torch.where((live & any_)[:, None], w[:, None] * grad, 0.0),
            "dP": dP, "size": size, "top": top, "any": any_, "p": p, "logp": logp,
            "sumP": P.abs().sum(0).max().item(), "sumZ": safe.abs().sum(0).max().item(), "gq": q @ P.abs() / T, "gp": pv @ P.abs() / T,
            "dq": (c.abs()[:, None] * qs).T @ safe.abs(), "dp": (c.abs()[:, None] * ps).T @ safe.abs()}


def bounds(ref, dt, r, N, k):
    """Absolute bounds of loss, lse, grad, dZ and dP."""
    es = (r + 2) * H32 * ref["size"]                       # a scaled score
    eq = 2 * es + 8 * H32 * (ref["top"] + 1) + 16 * H32     # q, relatively: score, lse, exponent, exponential
    log = ref["logp"].abs().amax(1)
    loss = 2 * es + 16 * H32 * (ref["top"] + log + 1) + 8 * H32 * (k + 1)
    lse = es + 16 * H32 * (ref["top"] + 1)
    step = 2.0 ** -8 if dt == "bf16" else 0.0              # half a step of the weights q
    pair = 2.0 ** -16 if dt == "bf16" else 0.0             # and of the teacher's weights, kept in two parts
    ep = (k + 16) * H32 * (1 + ref["top"])                 # p: exponent, exponential, sum
    many = 4096 * H32                                      # sums in fp32, over shares and blocks
    grad = (eq + step + many) * ref["gq"] + (ep + many) * ref["gp"]
    out = torch.finfo(DT[dt]).eps / 2
    # A weight c q below fp32's smallest normal number, 2^-126, may become 0: each of the N terms of an element of
    # dP is then off by up to 2^-126 |z| (and the V terms of one of grad by 2^-126 |P|), and the element itself, once
    # below 2^-126, by that. (Scores of hundreds give q of 1e-50, which the relative bounds alone cannot allow.)
    grad = grad + 2.0 ** -126 * (ref["sumP"] + 1)
    dP = (eq + step + many) * ref["dq"] + (ep + pair + many) * ref["dp"] + 2.0 ** -126 * (ref["sumZ"] + 1)
    dP = dP + out * (ref["dP"].abs() + dP)
    return {"loss": loss, "lse": lse, "grad": grad, "out": out, "dP": dP}


def inputs(N, V, r, k, dt, seed, T=1.0):
    g = torch.Generator().manual_seed(seed)
    P = (torch.randn(V, r, generator=g) * (2.5 / r ** 0.5)).to(DT[dt])
    Z = torch.randn(N, r, generator=g).to(DT[dt])
    idx = torch.randint(0, V, (N, k), generator=g, dtype=torch.int32)
    t = torch.randn(N, k, generator=g) * 3 * T
    w = torch.randn(N, generator=g)
    return Z.to(DEV), P.to(DEV), idx.to(DEV), t.to(DEV), w.to(DEV)


def check(Z, P, idx, t, w, T, dt):
    N, r = Z.shape
    k = idx.shape[1]
    loss, lse, grad = lr.distill(Z, P, idx, t, temperature=T)
    dZ, dP = lr.distill_grad(Z, P, idx, t, lse, grad, w, temperature=T)
    only, lse2, none = lr.distill(Z, P, idx, t, temperature=T, want_grad=False)
    torch.cuda.synchronize()
    assert none is None and dZ.dtype == Z.dtype and dP.dtype == P.dtype
    ref = reference(Z, P, idx, t, T, w)
    b = bounds(ref, dt, r, N, k)
    fine = torch.isfinite(Z).all(1).cpu()
    for name, got, want, tol in [("loss", loss, ref["loss"], b["loss"]), ("loss alone", only, ref["loss"], b["loss"]),
                                 ("lse", lse, ref["lse"], b["lse"]), ("lse alone", lse2, ref["lse"], b["lse"]),
                                 ("grad", grad, ref["grad"], b["grad"])]:
        err = (got.double().cpu() - want).abs()[fine]
        tol = (torch.zeros_like(want) + tol)[fine]
        assert bool((err <= tol).all()), f"{name}: {(err / tol).max().item():.3f} of its bound"
    wa = w.double().cpu().abs()[:, None]
    tol = wa * b["grad"]
    tol = tol + b["out"] * (ref["dZ"].abs() + tol) + H32 * ref["dZ"].abs()
    err = (dZ.double().cpu() - ref["dZ"]).abs()
    assert bool((err <= tol)[fine].all()), f"dZ: {(err - tol)[fine].max().item()}"
    err = (dP.double().cpu() - ref["dP"]).abs()
    assert bool((err <= b["dP"]).all()), f"dP: {(err / b['dP'].clamp(min=1e-300)).max().item():.3f} of its bound"
    return loss, lse, grad, dZ, dP


# ----------------------------------------------------------------- on the GPU

CASES = [
    # N, V, r, k: what it reaches
    (1, 1, 8, 1),          # one row, one token
    (1, 17, 8, 3),         # a vocabulary below one tile
    (5, 100, 16, 7),
    (32, 129, 32, 64),     # k above the tile, r = 32 exactly
    (33, 1000, 40, 5),     # one row past a 32-row tile, r padded to 64
    (64, 4099, 64, 64),
    (65, 4100, 72, 17),    # r padded to 128
    (127, 900, 128, 32),
    (128, 901, 128, 1),
    (129, 640, 136, 33),   # two waves of rows, r padded to 256
    (257, 5001, 256, 64),  # past one block of rows
    (31, 2500, 264, 9),    # r padded to 512
    (70, 1500, 512, 64),
    (300, 300, 504, 12),
    (1030, 257, 96, 20),   # many rows, few tokens: the columns pass splits the rows
    (700, 20011, 128, 48),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V,r,k", CASES)
def test_loss_and_gradients(N, V, r, k, dt):
    T = [1.0, 2.0, 0.5][(N + V) % 3]
    check(*inputs(N, V, r, k, dt, seed=N * 7 + V, T=T), T, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_empty_places_rows_and_repeated_ids(dt):
    N, V, r, k = 40, 700, 48, 11
    Z, P, idx, t, w = inputs(N, V, r, k, dt, seed=3)
    idx[0] = -1                       # nothing in the row
    t[1] = float("nan")               # the empty slots of fullhead_logits
    t[2] = float("-inf")
    idx[3, 2:] = -5
    idx[4, ::2] = V                   # just outside
    idx[5] = 2 ** 31 - 1
    idx[6] = 13                       # one id eleven times
    idx[7, 5:] = idx[7, :6].clone()
    t[8, 1:] = torch.finfo(torch.float32).min
    t[9, 3] = float("-inf")
    idx[10] = 0
    idx[11] = V - 1
    loss, lse, grad, dZ, dP = check(Z, P, idx, t, w, 1.0, dt)
    for row in (0, 1, 2, 5):
        assert loss[row] == 0 and not grad[row].any() and not dZ[row].any()
    assert bool(torch.isfinite(lse).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_masked_rows_do_not_reach_the_gradients(dt):
    """Rows without a place, and rows of weight 0, may hold anything."""
    N, V, r, k = 70, 900, 64, 8
    Z, P, idx, t, w = inputs(N, V, r, k, dt, seed=5)
    idx[3] = -1
    idx[50] = -1
    w[7] = 0
    w[69] = 0
    Z[3], Z[50] = float("nan"), float("inf")
    Z[7], Z[69] = float("inf"), float("nan")
    loss, lse, grad, dZ, dP = check(Z, P, idx, t, w, 1.0, dt)
    assert loss[3] == 0 and loss[50] == 0 and not dZ[[3, 50, 7, 69]].any()
    assert bool(torch.isfinite(dP).all())


@pytest.mark.gpu
def test_nan_of_a_weighted_row_shows():
    Z, P, idx, t, w = inputs(6, 300, 16, 4, "bf16", seed=1)
    Z[2] = float("nan")
    loss, lse, grad = lr.distill(Z, P, idx, t)
    assert bool(torch.isnan(loss[2])) and bool(torch.isfinite(loss[[0, 1, 3, 4, 5]]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt,scale", [("bf16", 40.0), ("fp32", 40.0), ("bf16", 0.0)])
def test_peaked_and_flat_students(dt, scale):
    """Scores of hundreds (every tile moves some row's maximum), and all equal."""
    Z, P, idx, t, w = inputs(50, 1200, 128, 16, dt, seed=9)
    check((Z.float() * scale).to(Z.dtype), P, idx, t, w, 1.0, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_frequent_ids(dt):
    """Every row names the same neighbouring ids: one group of columns holds all places."""
    N, V, r, k = 500, 3000, 128, 32
    Z, P, idx, t, w = inputs(N, V, r, k, dt, seed=11)
    idx[:] = torch.arange(k, dtype=torch.int32, device=DEV) + 64
    check(Z, P, idx, t, w, 1.0, dt)


@pytest.mark.gpu
def test_gradients_against_differences():
    """Central differences of the 64-bit loss along random directions, in fp32."""
    N, V, r, k = 12, 400, 24, 6
    Z, P, idx, t, w = inputs(N, V, r, k, "fp32", seed=21)
    loss, lse, grad = lr.distill(Z, P, idx, t)
    dZ, dP = lr.distill_grad(Z, P, idx, t, lse, grad, w)
    ref = reference(Z, P, idx, t, 1.0, w)
    b = bounds(ref, "fp32", r, N, k)
    wd = w.double().cpu()
    value = lambda z, p: (wd * reference(z, p, idx, t, 1.0, w)["loss"]).sum()  # noqa: E731
    g = torch.Generator().manual_seed(4)
    h = 1e-5
    for _ in range(3):
        a = torch.randn(N, r, generator=g, dtype=torch.float64)
        c = torch.randn(V, r, generator=g, dtype=torch.float64)
        z, p = Z.double().cpu(), P.double().cpu()
        num = (value(z + h * a, p + h * c) - value(z - h * a, p - h * c)) / (2 * h)
        got = (dZ.double().cpu() * a).sum() + (dP.double().cpu() * c).sum()
        tol = ((wd.abs()[:, None] * b["grad"] + H32 * 2 * ref["dZ"].abs()) * a.abs()).sum() + (b["dP"] * c.abs()).sum()
        # the differences: h^2 times a third derivative of the order of |direction . scores|^3, and 2^-52 / h
        cube = (a.abs() @ P.double().cpu().abs().T + z.abs() @ c.abs().T).max() ** 3 * wd.abs().sum()
        assert abs(num - got) <= tol + h * h * cube + 2.0 ** -50 / h * wd.abs().sum() * 20


@pytest.mark.gpu
def test_autograd_gives_the_calls_gradients():
    Z, P, idx, t, w = inputs(37, 800, 64, 9, "bf16", seed=2)
    loss, lse, grad = lr.distill(Z, P, idx, t, temperature=2.0)
    dZ, dP = lr.distill_grad(Z, P, idx, t, lse, grad, w, temperature=2.0)
    z, p = Z.clone().requires_grad_(), P.clone().requires_grad_()
    out = lr.distill_loss(z, p, idx, t, temperature=2.0)
    assert torch.equal(out.detach(), loss)
    (out * w).sum().backward()
    assert torch.equal(z.grad, dZ) and torch.equal(p.grad, dP)
    z2 = Z.clone().requires_grad_()
    gz, = torch.autograd.grad(lr.distill_loss(z2, P, idx, t, temperature=2.0), z2, w)
    assert torch.equal(gz, dZ)
    p2 = P.clone().requires_grad_()
    gp, = torch.autograd.grad(lr.distill_loss(Z, p2, idx, t, temperature=2.0), p2, w)
    assert torch.equal(gp, dP)
    # an expanded gradient, as that of a sum
    gs, = torch.autograd.grad(lr.distill_loss(z2, P, idx, t, temperature=2.0).sum(), z2)
    assert torch.equal(gs, lr.distill_grad(Z, P, idx, t, lse, grad, temperature=2.0)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dt,N,r,k", [
    ("bf16", 700, 32, 64), ("bf16", 700, 64, 64), ("bf16", 701, 128, 64), ("bf16", 300, 256, 63), ("bf16", 200, 512, 64),
    ("bf16", 64, 128, 64), ("bf16", 33, 512, 64), ("fp32", 150, 40, 64),
])
@pytest.mark.parametrize("span", [1, 20, 400])
def test_frequent_tokens(dt, N, r, k, span):
    """Most rows name the same few tokens (with span 1, the same one k times over)."""
    Z, P, idx, t, w = inputs(N, 1500, r, k, dt, seed=N + span)
    idx = 100 + idx % span
    idx[:, -1] = torch.arange(N, dtype=torch.int32, device=DEV) % 1500
    check(Z, P, idx.contiguous(), t, w, 1.0, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_micro_batches_of_odd_sizes(dt):
    """Views that start off 16 bytes, forward and backward: the rows' own
    results do not depend on where the batch is cut."""
    Z, P, idx, t, w = inputs(45, 700, 32, 5, dt, seed=14)
    loss, lse, grad = lr.distill(Z, P, idx, t)
    want = lr.distill_grad(Z[7:], P, idx[7:], t[7:], lse[7:], grad[7:], w[7:])
    same = lr.distill_grad(Z[7:].clone(), P, idx[7:].clone(), t[7:].clone(), lse[7:].clone(), grad[7:].clone(),
                           w[7:].clone())
    assert all(torch.equal(a, b) for a, b in zip(want, same))
    z = Z.clone().requires_grad_()
    whole = torch.cat([lr.distill_loss(z[:7], P, idx[:7], t[:7]), lr.distill_loss(z[7:], P, idx[7:], t[7:])])
    (whole * w).sum().backward()          # the second part's gradient is a view from element 7 on
    ref = reference(Z, P, idx, t, 1.0, w)
    b = bounds(ref, dt, 32, 45, 5)
    assert bool(((whole.detach().double().cpu() - ref["loss"]).abs() <= b["loss"]).all())
    tol = b["grad"] * w.double().cpu().abs()[:, None]
    tol = tol + b["out"] * (ref["dZ"].abs() + tol) + H32 * 2 * ref["dZ"].abs()
    assert bool(((z.grad.double().cpu() - ref["dZ"]).abs() <= tol).all())


@pytest.mark.gpu
def test_either_gradient_alone_and_no_rows():
    Z, P, idx, t, w = inputs(20, 500, 32, 4, "bf16", seed=6)
    loss, lse, grad = lr.distill(Z, P, idx, t)
    dZ, dP = lr.distill_grad(Z, P, idx, t, lse, grad, w)
    z_only, none = lr.distill_grad(Z, P, idx, t, lse, grad, w, want_dP=False)
    assert none is None and torch.equal(z_only, dZ)
    none, p_only = lr.distill_grad(Z, P, idx, t, lse, None, w, want_dZ=False)
    assert none is None and torch.equal(p_only, dP)
    e = lr.distill(Z[:0], P, idx[:0], t[:0])
    assert [tuple(x.shape) for x in e] == [(0,), (0,), (0, 32)]
    dZ0, dP0 = lr.distill_grad(Z[:0], P, idx[:0], t[:0], e[1], e[2])
    assert dZ0.shape == (0, 32) and not dP0.any()


@pytest.mark.gpu
@pytest.mark.parametrize("dt,N,r", [("bf16", 300, 128), ("bf16", 3, 512), ("fp32", 40, 64)])
def test_graph_replays_match_eager_calls(dt, N, r):
    V, k = 3000, 16
    sets = [inputs(N, V, r, k, dt, seed=s) for s in (31, 32, 33)]
    eager = []
    for Z, P, idx, t, w in sets:
        loss, lse, grad = lr.distill(Z, P, idx, t)
        eager.append((loss, *lr.distill_grad(Z, P, idx, t, lse, grad, w)))
    held = [x.clone() for x in sets[0]]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):   # two graphs over the same inputs
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            loss, lse, grad = lr.distill(*held[:4])
            dZ, dP = lr.distill_grad(*held[:4], lse, grad, held[4])
        graphs.append((g, (loss, dZ, dP)))
    for s, want in list(zip(sets, eager)) + [(sets[1], eager[1])]:
        for x, y in zip(held, s):
            x.copy_(y)
        for g, out in graphs:
            for o in out:
                o.fill_(float("nan"))
            g.replay()
        lr.distill(*s[:4])   # the program's own work between the replays
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_autograd_refuses_capture():
    Z, P, idx, t, _ = inputs(8, 200, 16, 4, "bf16", seed=1)
    Z.requires_grad_()
    lr.distill_loss(Z, P, idx, t).sum().backward()
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="cannot be captured"):
        with torch.cuda.graph(g):
            lr.distill_loss(Z, P, idx, t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.no_grad():   # without gradients it can
        with torch.cuda.graph(g):
            out = lr.distill_loss(Z, P, idx, t)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, lr.distill(Z.detach(), P, idx, t)[0])


@pytest.mark.gpu
def test_side_stream_and_repeats_are_bitwise_equal():
    Z, P, idx, t, w = inputs(257, 7001, 128, 64, "bf16", seed=17)
    loss, lse, grad = lr.distill(Z, P, idx, t)
    want = (loss, *lr.distill_grad(Z, P, idx, t, lse, grad, w))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = []
    with torch.cuda.stream(s):
        for _ in range(3):
            loss, lse, grad = lr.distill(Z, P, idx, t)
            got.append((loss, *lr.distill_grad(Z, P, idx, t, lse, grad, w)))
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
@pytest.mark.timeout(300)
def test_offsets_past_32_bits():
    """A head of 4.3 GB: the rows behind 2^32 bytes take part, and get their gradient."""
    V, r, N, k = (1 << 22) + 77, 512, 3, 4
    g = torch.Generator(device=DEV).manual_seed(8)
    P = torch.randn(V, r, generator=g, device=DEV, dtype=torch.bfloat16) * 0.1
    Z = torch.randn(N, r, generator=g, device=DEV).bfloat16()
    idx = torch.tensor([[V - 1, 0, 5, V - 77], [V - 2, 1, 2, 3], [V - 3, V - 4, 7, 9]], dtype=torch.int32, device=DEV)
    t = torch.randn(N, k, generator=g, device=DEV)
    loss, lse, grad = lr.distill(Z, P, idx, t)
    _, dP = lr.distill_grad(Z, P, idx, t, lse, grad, want_dZ=False)
    s = torch.cat([Z.double() @ c.double().T for c in P.split(1 << 19)], 1)
    ref = torch.logsumexp(s, 1)
    es = (r + 2) * H32 * float((Z.double().abs() @ P[:4096].double().abs().T).max()) * 2
    assert bool(((lse - ref).abs() <= es + 16 * H32 * (ref.abs() + s.abs().amax(1) + 1)).all())
    rows = torch.cat([torch.arange(8), torch.arange(V - 90, V)]).to(DEV)
    q = torch.exp(s[:, rows] - ref[:, None])
    p = torch.zeros(N, V, dtype=torch.float64, device=DEV).scatter_add_(1, idx.long(), torch.softmax(t.double(), 1))
    want = (q - p[:, rows]).T @ Z.double()
    size = (q + p[:, rows]).T @ Z.double().abs()
    err = (dP[rows].double() - want).abs()
    assert bool((err <= (2.0 ** -8 * 2.1 + 4 * es) * size).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bf16"])
def test_training_steps_on_a_factored_head(dt):
    """The operators as they are used: the full head's top logits teach a head
    made by factor(); the step's gradients are those of the definition."""
    V, d, r, N, k = 3000, 256, 32, 48, 16
    inp = gen.make_custom(V, d, r, N, dt, seed=77)
    W, H, Q, P = (dev(inp[x], DEV) for x in ("W", "H", "Q", "P"))
    omega = torch.from_numpy(np.random.default_rng(1).standard_normal((d, r)).astype(np.float32)).to(DEV)
    P, Q = lr.factor(W, r, omega)
    for _ in range(2):
        head = lr.Head(Q, P, W, B_max=N, k_max=k)
        ids, logits = head.full_topk(H, k)
        q, p = Q.float().requires_grad_(), P.clone().requires_grad_()
        Z = (H.float() @ q.T).bfloat16()
        Z.retain_grad()
        lr.distill_loss(Z, p, ids, logits, temperature=2.0).mean().backward()
        w = torch.full((N,), 1.0 / N, device=DEV)
        ref = reference(Z.detach(), P, ids, logits, 2.0, w)
        b = bounds(ref, dt, r, N, k)
        assert bool(((p.grad.double().cpu() - ref["dP"]).abs() <= b["dP"]).all())
        tol = b["grad"] / N
        tol = tol + b["out"] * (ref["dZ"].abs() + tol) + H32 * 2 * ref["dZ"].abs()
        assert bool(((Z.grad.double().cpu() - ref["dZ"]).abs() <= tol).all())
        assert q.grad.shape == Q.shape and bool(torch.isfinite(q.grad).all())
        P = (P.float() - 0.1 * p.grad.float()).bfloat16()
        Q = (Q.float() - 0.1 * q.grad).bfloat16()
    idx, score, exact = lr.Head(Q, P, W, B_max=N, k_max=k).draft(H, k)
    torch.cuda.synchronize()
    assert bool((idx >= 0).all()) and bool(torch.isfinite(exact).all())
