"""Refusals of sampling, verification and the embedding, before anything is
launched (stand-in addresses, never dereferenced)."""
import ctypes

import pytest
import torch

import rank_lm_head_amd as lr
from rank_lm_head_amd import _lib
from rank_lm_head_amd._lib import BF16, EALIGN, EDTYPE, EINVAL, ERANGE, EWORKSPACE, FP32, OK

A = 0x100000
HOW = _lib.Sampling(None, None, None, None, 1.0, 0, 1.0, 0.0)


def how(**ptrs):
    return _lib.Sampling(*[ptrs.get(k) for k in ("temperature", "top_k", "top_p", "min_p")], 1.0, 0, 1.0, 0.0)


def sample(dtype=FP32, logits=A, ld=1000, idx=None, u=A, how=HOW, B=2, n=1000, token=A, prob=A, probs=None, ws=A,
           nbytes=1 << 40):
    return _lib.load().lrhead_sample(dtype, logits, ld, idx, u, how, B, n, token, prob, probs, ws, nbytes, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=2), EDTYPE), (dict(n=0, ld=8), ERANGE), (dict(n=2 ** 24 + 1, ld=2 ** 25), ERANGE), (dict(ld=999), ERANGE),
    (dict(B=-1), ERANGE), (dict(B=2 ** 20 + 1), ERANGE), (dict(B=2 ** 20, n=2 ** 24, ld=2 ** 24), ERANGE),
    (dict(probs=A), ERANGE), (dict(logits=None), EINVAL), (dict(u=None), EINVAL), (dict(how=None), EINVAL),
    (dict(token=None), EINVAL), (dict(ws=None), EINVAL), (dict(logits=A + 2), EALIGN), (dict(dtype=BF16, logits=A + 1), EALIGN),
    (dict(u=A + 2), EALIGN), (dict(idx=A + 1), EALIGN), (dict(token=A + 4), EALIGN), (dict(prob=A + 8), EALIGN),
    (dict(n=64, ld=64, probs=A + 4), EALIGN), (dict(ws=A + 8), EALIGN), (dict(nbytes=16), EWORKSPACE),
    (dict(n=64, ld=64, nbytes=16), EWORKSPACE),
    (dict(how=how(temperature=A + 1)), EALIGN), (dict(how=how(top_k=A + 2)), EALIGN), (dict(how=how(top_p=A + 3)), EALIGN),
    (dict(how=how(min_p=A + 1)), EALIGN), (dict(B=0, logits=None, ws=None), OK), (dict(B=0, ld=999), ERANGE),
])
def test_sample(kwargs, code):
    assert sample(**kwargs) == code
    if code:
        assert _lib.load().lrhead_last_error()


def verify(dtype=FP32, logits=A, ld=1000, token=A, idx=A, probs=A, k=8, length=None, u=A, how=HOW, B=2, s=3, n=1000,
           out=A, count=A, ws=A, nbytes=1 << 40):
    return _lib.load().lrhead_verify(dtype, logits, ld, token, idx, probs, k, length, u, how, B, s, n, out, count, ws,
                                     nbytes, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=-1), EDTYPE), (dict(s=-1), ERANGE), (dict(s=256), ERANGE), (dict(n=0), ERANGE), (dict(ld=5), ERANGE),
    (dict(B=2 ** 18 + 1), ERANGE), (dict(B=-1), ERANGE), (dict(k=0), ERANGE), (dict(k=65), ERANGE),
    (dict(probs=None), EINVAL), (dict(idx=None), EINVAL), (dict(logits=None), EINVAL), (dict(token=None), EINVAL),
    (dict(u=None), EINVAL), (dict(how=None), EINVAL), (dict(out=None), EINVAL), (dict(count=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(token=A + 1), EALIGN), (dict(idx=A + 2), EALIGN), (dict(probs=A + 2), EALIGN),
    (dict(length=A + 2), EALIGN), (dict(out=A + 4), EALIGN), (dict(count=A + 4), EALIGN), (dict(ws=A + 4), EALIGN),
    (dict(nbytes=100), EWORKSPACE), (dict(B=0, ws=None, logits=None), OK),
])
def test_verify(kwargs, code):
    assert verify(**kwargs) == code


def embed(dtype=FP32, W=A, V=100, d=8, token=0x900000, N=4, scale=1.0, out=0x800000):
    return _lib.load().lrhead_embed(dtype, W, V, d, token, N, scale, out, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=9), EDTYPE), (dict(V=0), ERANGE), (dict(V=2 ** 31), ERANGE), (dict(d=0), ERANGE), (dict(d=65537), ERANGE),
    (dict(N=-1), ERANGE), (dict(N=2 ** 20 + 1), ERANGE), (dict(N=2 ** 20, d=65536), ERANGE), (dict(scale=float("nan")), ERANGE),
    (dict(scale=float("inf")), ERANGE), (dict(W=None), EINVAL), (dict(token=None), EINVAL), (dict(out=None), EINVAL),
    (dict(W=A + 2), EALIGN), (dict(out=0x800001), EALIGN), (dict(token=0x900002), EALIGN), (dict(out=A + 64), EINVAL),
    (dict(token=0x800010), EINVAL), (dict(N=0, W=None), OK),
])
def test_embed(kwargs, code):
    assert embed(**kwargs) == code


def embed_grad(dtype=FP32, dY=A, token=0x900000, N=4, V=100, d=8, scale=1.0, add=0, dW=0x800000, ws=0xa00000,
               nbytes=1 << 40):
    return _lib.load().lrhead_embed_grad(dtype, dY, token, N, V, d, scale, add, dW, ws, nbytes, None)


@pytest.mark.parametrize("kwargs,code", [
    (dict(dtype=9), EDTYPE), (dict(V=0), ERANGE), (dict(d=65537), ERANGE), (dict(N=2 ** 20 + 1), ERANGE),
    (dict(scale=float("nan")), ERANGE), (dict(dY=None), EINVAL), (dict(token=None), EINVAL), (dict(dW=None), EINVAL),
    (dict(ws=None), EINVAL), (dict(dY=A + 1), EALIGN), (dict(dW=A + 2), EALIGN), (dict(token=0x900002), EALIGN),
    (dict(ws=0xa00008), EALIGN), (dict(nbytes=64), EWORKSPACE), (dict(dW=A + 32), EINVAL), (dict(token=0x800010), EINVAL),
    (dict(N=0, add=1, dY=None, ws=None, token=None), OK),
])
def test_embed_grad(kwargs, code):
    assert embed_grad(**kwargs) == code


def test_workspace_bytes_are_host_arithmetic():
    lib = _lib.load()
    assert lib.lrhead_sample_workspace_bytes(FP32, 256, 151936) >= 256 * 75 * (8 + 4 + 32)
    assert lib.lrhead_sample_workspace_bytes(BF16, 0, 1) > 0
    assert lib.lrhead_sample_workspace_bytes(BF16, 1, 0) == 0 and lib.lrhead_sample_workspace_bytes(5, 1, 9) == 0
    assert lib.lrhead_verify_workspace_bytes(BF16, 4, 255, 151936) > lib.lrhead_verify_workspace_bytes(BF16, 4, 0, 151936) > 0
    assert lib.lrhead_verify_workspace_bytes(BF16, 4, 256, 100) == 0 and lib.lrhead_verify_workspace_bytes(BF16, -1, 2, 9) == 0
    assert lib.lrhead_embed_grad_workspace_bytes(FP32, 100, 8, 5000) > 5000 * 8
    assert lib.lrhead_embed_grad_workspace_bytes(FP32, 100, 8, 50) > 0
    assert lib.lrhead_embed_grad_workspace_bytes(FP32, 100, 0, 50) == 0 and lib.lrhead_embed_grad_workspace_bytes(FP32, 9, 8, 0) > 0


def test_bindings_refuse_cpu_tensors_and_settings_that_do_not_fit():
    f, i = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="device tensor"):
        lr.sample(f(2, 8), f(2))
    with pytest.raises(ValueError, match="device tensor"):
        lr.verify(f(2, 3, 8), i(2, 2), f(2, 3))
    with pytest.raises(ValueError, match="device matrix"):
        lr.embed(f(5, 8), i(3))
    with pytest.raises(ValueError, match="device tensor"):
        lr.embed_grad(f(3, 8), i(3), 5)
    for W in (f(5, 8), f(5, 8, requires_grad=True)):
        with pytest.raises(ValueError, match="device matrix"):
            lr.embedding(W, i(3))


def test_embedding_refuses_forward_mode():
    import torch.autograd.forward_ad as fw
    with fw.dual_level():
        W = fw.make_dual(torch.zeros(5, 8), torch.ones(5, 8))
        with pytest.raises(NotImplementedError, match="forward"):
            lr.embedding(W, torch.zeros(3, dtype=torch.int32))
        with torch.no_grad(), pytest.raises(NotImplementedError, match="forward"):
            lr.embedding(W, torch.zeros(3, dtype=torch.int32))


@pytest.mark.gpu
def test_bindings_refuse_what_does_not_fit_together():
    dev = "cuda:0"
    f = lambda *s, **k: torch.zeros(*s, device=dev, **k)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    x = f(2, 100)
    for bad in [dict(u=f(3)), dict(u=f(2).double()), dict(u=torch.zeros(2)), dict(idx=i(2, 99)), dict(idx=f(2, 100)),
                dict(temperature=f(3)), dict(temperature=i(2)), dict(top_k=f(2)), dict(top_k=2 ** 31), dict(top_p=f(2, 1)),
                dict(min_p=torch.zeros(2)), dict(want_probs=True), dict(logits=f(2, 100).half()), dict(logits=f(100)),
                dict(logits=f(100, 2).t()), dict(logits=f(1, 100).expand(2, 100)), dict(logits=f(2, 0))]:
        with pytest.raises(ValueError):
            lr.sample(bad.pop("logits", x), bad.pop("u", f(2)), **bad)
    x = f(2, 4, 100)
    for bad in [dict(token=i(2, 4)), dict(token=f(2, 3)), dict(u=f(2, 3)), dict(idx=i(2, 3, 8)), dict(probs=f(2, 3, 8)),
                dict(idx=i(2, 3, 8), probs=f(2, 3, 7)), dict(idx=i(6, 8), probs=f(6, 8)), dict(length=i(3)), dict(length=f(2)),
                dict(logits=f(8, 100)), dict(logits=f(4, 2, 100).transpose(0, 1)), dict(logits=f(2, 0, 100)), dict(top_p=f(8))]:
        with pytest.raises(ValueError):
            lr.verify(bad.pop("logits", x), bad.pop("token", i(2, 3)), bad.pop("u", f(2, 4)), **bad)
    with pytest.raises(lr.LrheadError):
        lr.verify(x, i(2, 3), f(2, 4), idx=i(2, 3, 65), probs=f(2, 3, 65))
    for bad in [(f(5, 8), f(3)), (f(5, 8).t(), i(3)), (f(5, 8), i(6)[::2]), (f(5, 8), torch.zeros(3, dtype=torch.int32)),
                (f(5), i(3))]:
        with pytest.raises(ValueError):
            lr.embed(*bad)
    with pytest.raises(ValueError):
        lr.embed(f(5, 8), i(3), scale=float("nan"))
    y = f(3, 8)
    for bad in [dict(token=i(4)), dict(token=f(3)), dict(V=0), dict(V=2 ** 31), dict(out=f(5, 7)), dict(out=f(5, 8).bfloat16()),
                dict(out=f(8, 5).t()), dict(dY=f(8, 3).t()), dict(dY=f(3, 8).half()), dict(scale=float("inf"))]:
        with pytest.raises(ValueError):
            lr.embed_grad(bad.pop("dY", y), bad.pop("token", i(3)), bad.pop("V", 5), **bad)


APART = [0x1000000 * (i + 1) for i in range(16)]   # stand-ins with 16 MiB between them


@pytest.mark.parametrize("a,b", [(o, i) for o in ("token", "prob", "probs", "ws") for i in
                                 ("logits", "idx", "u", "temperature", "top_k", "top_p", "min_p", "token", "prob", "probs",
                                  "ws") if o != i])
def test_sample_refuses_outputs_over_inputs(a, b):
    names = ["logits", "idx", "u", "temperature", "top_k", "top_p", "min_p", "token", "prob", "probs", "ws"]
    at = dict(zip(names, APART))
    at[a] = at[b]
    settings = {k: at.pop(k) for k in ("temperature", "top_k", "top_p", "min_p")}
    assert sample(**at, n=64, ld=64, B=9, how=how(**settings)) == EINVAL


def test_sample_refuses_an_output_among_the_last_row_s_logits():
    at = dict(logits=APART[0], u=APART[1], token=APART[2], prob=APART[3], ws=APART[4])
    assert sample(**{**at, "token": APART[0] + 4 * (2 * 2000 + 996)}, ld=2000, B=3, n=1000) == EINVAL
    assert sample(**{**at, "ws": APART[0] + 4 * (2 * 2000 + 996)}, ld=2000, B=3, n=1000) == EINVAL


@pytest.mark.parametrize("a,b", [(o, i) for o in ("out", "count", "ws") for i in
                                 ("logits", "token", "idx", "probs", "length", "u", "temperature", "top_k", "top_p", "min_p",
                                  "out", "count", "ws") if o != i])
def test_verify_refuses_outputs_over_inputs(a, b):
    names = ["logits", "token", "idx", "probs", "length", "u", "temperature", "top_k", "top_p", "min_p", "out", "count", "ws"]
    at = dict(zip(names, APART))
    at[a] = at[b]
    settings = {k: at.pop(k) for k in ("temperature", "top_k", "top_p", "min_p")}
    assert verify(**at, B=9, how=how(**settings)) == EINVAL


@pytest.mark.parametrize("a,b", [("dW", "dY"), ("dW", "token"), ("dW", "ws"), ("ws", "dY"), ("ws", "token")])
def test_embed_grad_refuses_outputs_over_inputs(a, b):
    at = dict(zip(["dY", "token", "dW", "ws"], APART))
    at[a] = at[b]
    assert embed_grad(**at) == EINVAL
