"""Distillation where the student is close to its teacher: the gradients are
sums of q - p, small differences of the teacher's places' large terms.

The bounds count the roundings of tests/test_distill.py, but for one: at a
teacher's place, what the rounding of q to bf16 takes away is made good, so
only the other tokens' q counts half a step of bf16 (2^-8 of it).
"""
import pytest
import torch

import rank_lm_head_amd as lr
from test_distill import DEV, DT, H32

BF = torch.bfloat16


def definition(Z, P, idx, t, T, w):
    """grad, dP, and what their bounds are made of, in 64 bits."""
    N, V = Z.shape[0], P.shape[0]
    Z, P, t, w = Z.double(), P.double(), t.double(), w.double()
    s = Z @ P.T / T
    lse = torch.logsumexp(s, 1)
    q = torch.exp(s - lse[:, None])
    logp = torch.log_softmax(t / T, 1)
    p = torch.zeros_like(q).scatter_add_(1, idx.long(), torch.exp(logp))
    place = torch.zeros_like(q).scatter_(1, idx.long(), 1.0)
    c = w / T
    return {"grad": (q - p) @ P / T, "dP": (c[:, None] * (q - p)).T @ Z,
            "gq": q @ P.abs() / T, "gp": p @ P.abs() / T, "go": (q * (1 - place)) @ P.abs() / T,
            "dq": (c.abs()[:, None] * q).T @ Z.abs(), "dp": (c.abs()[:, None] * p).T @ Z.abs(),
            "do": (c.abs()[:, None] * q * (1 - place)).T @ Z.abs(),
            "size": (Z.abs() @ P.abs().T).max().item() / T, "top": s.abs().max().item() + lse.abs().max().item(),
            "sumP": P.abs().sum(0).max().item(), "sumZ": Z.abs().sum(0).max().item(), "q": q, "p": p}


def check(Z, P, idx, t, w, T, dt="bf16"):
    (N, r), k = Z.shape, idx.shape[1]
    loss, lse, grad = lr.distill(Z, P, idx, t, temperature=T)
    dZ, dP = lr.distill_grad(Z, P, idx, t, lse, grad, w, temperature=T)
    d = definition(Z, P, idx, t, T, w)
    es = (r + 2) * H32 * d["size"]                          # a scaled score
    eq = 2 * es + 8 * H32 * (d["top"] + 1) + 16 * H32       # q, relatively: score, lse, exponent, exponential
    ep = (k + 16) * H32 * (1 + d["top"])                    # p: exponent, exponential, sum
    many = 4096 * H32                                       # sums in fp32, over shares and blocks
    step = 2.0 ** -8 if dt == "bf16" else 0.0               # half a step of q, away from the places
    pair = 2.0 ** -16 if dt == "bf16" else 0.0              # the places' weights, kept in two parts
    out = torch.finfo(DT[dt]).eps / 2
    tol = (eq + many) * d["gq"] + step * d["go"] + (ep + many) * d["gp"] + 2.0 ** -126 * (d["sumP"] + 1)
    err = (grad.double() - d["grad"]).abs()
    assert bool((err <= tol).all()), f"grad: {(err / tol).max().item():.3f} of its bound"
    wa = w.double()[:, None]
    tol = wa.abs() * tol
    tol = tol + out * ((wa * d["grad"]).abs() + tol) + H32 * (wa * d["grad"]).abs()
    err = (dZ.double() - wa * d["grad"]).abs()
    assert bool((err <= tol).all()), f"dZ: {(err / tol).max().item():.3f} of its bound"
    # a place's weight is at most p and the rounding of q, 2^-8 of it
    tol = ((eq + many) * d["dq"] + step * d["do"] + (ep + many + pair) * d["dp"] + pair * 2.0 ** -8 * d["dq"]
           + 2.0 ** -126 * (d["sumZ"] + 1))
    tol = tol + out * (d["dP"].abs() + tol)
    err = (dP.double() - d["dP"]).abs()
    assert bool((err <= tol).all()), f"dP: {(err / tol).max().item():.3f} of its bound"
    return d, loss, grad, dZ, dP


def student(N, V, r, seed, sharp, dt="bf16"):
    g = torch.Generator().manual_seed(seed)
    P = (torch.randn(V, r, generator=g) * (2.5 / r ** 0.5)).to(DT[dt]).to(DEV)
    Z = (torch.randn(N, r, generator=g) * sharp).to(DT[dt]).to(DEV)
    return Z, P, torch.randn(N, generator=g).to(DEV), g


def teacher_of(Z, P, k, g, noise=1e-3):
    """The student's own best k tokens, their scores off by a little noise, in no order."""
    top = (Z.double() @ P.double().T).topk(k, 1)
    t = top.values.float() + noise * torch.randn(Z.shape[0], k, generator=g).to(DEV)
    mix = torch.rand(Z.shape[0], k, generator=g).to(DEV).argsort(1)
    return top.indices.gather(1, mix).int().contiguous(), t.gather(1, mix).contiguous()


@pytest.mark.gpu
@pytest.mark.parametrize("N,V,r,k,T", [
    (20, 5000, 32, 16, 1.0),       # four waves share a row's tiles
    (20, 5000, 200, 40, 1.0),      # two do, r padded
    (50, 5000, 128, 16, 2.0),
    (64, 3000, 512, 64, 1.0),
    (65, 3000, 512, 64, 1.0),      # a row past the columns pass for few rows
    (300, 5000, 32, 16, 1.0),
    (300, 5000, 56, 33, 0.5),
    (300, 5000, 128, 32, 1.0),
    (150, 3000, 256, 64, 1.0),
    (130, 3001, 504, 7, 1.0),
    (700, 20011, 128, 48, 1.0),    # several tiles a share
])
def test_gradients_near_agreement(N, V, r, k, T):
    Z, P, w, g = student(N, V, r, N + r, 2.0 * T)
    idx, t = teacher_of(Z, P, k, g)
    d, loss, *_ = check(Z, P, idx, t, w, T)
    # it is what it claims to be: peaked students, little loss
    assert d["q"].amax(1).mean() > 0.3 and loss.mean() < 0.3


@pytest.mark.gpu
@pytest.mark.parametrize("N,r", [(40, 64), (300, 64), (300, 128), (90, 304)])
def test_an_id_that_occurs_twice_near_agreement(N, r):
    """Its two places share the token's probability; q is there once."""
    Z, P, w, g = student(N, 4000, r, r, 2.0)
    idx, t = teacher_of(Z, P, 8, g)
    idx = torch.cat([idx, idx[:, 2:5]], 1).contiguous()
    half = torch.log(torch.tensor(2.0, dtype=torch.float64))
    t = t.double()
    t[:, 2:5] -= half
    t = torch.cat([t, t[:, 2:5]], 1).float().contiguous()
    check(Z, P, idx, t, w, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("N,r", [(600, 32), (600, 128), (300, 256), (200, 512)])
def test_one_teacher_for_all_rows_near_agreement(N, r):
    """Rows that differ little name the same few tokens, whose places are summed ahead."""
    Z, P, w, g = student(N, 3000, r, N + r, 0.05)
    Z = (Z.float() + 2.0 * torch.randn(r, generator=g).to(DEV)).to(BF)
    idx, t = teacher_of(Z, P, 32, g)
    check(Z, P, idx, t, w, 1.0)


@pytest.mark.gpu
def test_fp32_near_agreement():
    Z, P, w, g = student(100, 3000, 64, 5, 2.0, "fp32")
    idx, t = teacher_of(Z, P, 16, g)
    check(Z, P, idx, t, w, 1.0, "fp32")
