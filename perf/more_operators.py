"""Timed cases of a drafter's token loop: sampling, verification of drafted tokens, embedding.

sample:      a token of each row of logits under temperature, top-k, top-p and min-p, from given uniform numbers.
verify:      drafted tokens accepted or replaced so that what comes out is distributed as the target's own samples.
embed:       the rows of an embedding matrix at given tokens, scaled.
embed_grad:  the gradient of that matrix.

`run` computes a case in its plain form (torch operations in 32 bits, in 64 where a random number is held against
sums of probabilities), or, with `own` set, through the package.
"""
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
V0 = 151936          # vocabulary of the drafter head
# settings that the requests of one batch bring along: temperature, top_k, top_p, min_p
MIXED = [(0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0), (0.6, 20, 0.95, 0.0), (0.8, 0, 0.9, 0.0), (0.7, 50, 1.0, 0.0),
         (1.0, 0, 1.0, 0.05), (1.2, 200, 0.98, 0.02)]


def listed():
    s = lambda name, **c: {"name": name, "op": "sample", **c}  # noqa: E731
    v = lambda name, **c: {"name": name, "op": "verify", **c}  # noqa: E731
    e = lambda name, **c: {"name": name, "op": "embed", **c}  # noqa: E731
    g = lambda name, **c: {"name": name, "op": "embed_grad", **c}  # noqa: E731
    return [
        # one request decoding over the full head's fp32 logits with usual settings: latency
        s("sample_1_top20", B=1, n=V0, dtype="fp32", lists=False, mixed=False, T=0.6, k=20, p=0.95, m=0.0),
        # a batch of 64 requests under nucleus sampling alone, a bf16 head's logits
        s("sample_64_nucleus", B=64, n=V0, dtype="bf16", lists=False, mixed=False, T=0.8, k=0, p=0.9, m=0.0),
        # a serving batch whose requests bring their own settings, greedy ones among them
        s("sample_256_mixed", B=256, n=V0, dtype="fp32", lists=False, mixed=True, T=1.0, k=0, p=1.0, m=0.0),
        # samples of the distribution as it is (policy rollouts), odd vocabulary and batch
        s("sample_33_odd", B=33, n=32003, dtype="fp32", lists=False, mixed=False, T=1.0, k=0, p=1.0, m=0.0),
        # a drafter's step: candidate lists of 256 rows, with the distribution that verification needs
        s("sample_lists_256x32", B=256, n=32, dtype="fp32", lists=True, mixed=False, T=0.8, k=0, p=1.0, m=0.0),
        # one request, five drafted tokens: latency
        v("verify_1x5", B=1, s=5, n=V0, k=32, dtype="fp32", mixed=False, T=0.6, top_k=20, p=0.95, m=0.0, ragged=False),
        # 32 requests with up to seven drafted tokens each and settings of their own
        v("verify_32x7_mixed", B=32, s=7, n=V0, k=32, dtype="bf16", mixed=True, T=1.0, top_k=0, p=1.0, m=0.0, ragged=True),
        # one token of each of 256 requests
        e("embed_256", N=256, V=V0, d=5120, dtype="bf16", scale=1.0),
        # a prefill or training batch of 16384 positions, scaled by sqrt(d)
        e("embed_16384_scaled", N=16384, V=V0, d=5120, dtype="bf16", scale=5120 ** 0.5),
        # a training step on one sequence of 4096 positions, odd vocabulary
        g("embed_grad_4096x5120", N=4096, V=32003, d=5120, dtype="bf16", scale=1.0),
        # four sequences, narrower rows, the large vocabulary
        g("embed_grad_16384x1024", N=16384, V=V0, d=1024, dtype="bf16", scale=32.0),
        # the tiny fp32 model
        g("embed_grad_tiny_fp32", N=333, V=4096, d=256, dtype="fp32", scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["sample", "sample", "verify", "embed", "embed_grad"])
    dtype = rng.choice(["bf16", "fp32"])
    how = {"mixed": rng.random() < 0.3, "T": rng.choice([1.0, 0.6, 0.8, 1.3]), "p": rng.choice([1.0, 1.0, 0.9, 0.95]),
           "m": rng.choice([0.0, 0.0, 0.05])}
    top_k = rng.choice([0, 0, _log(rng, 1, 400)])
    if op == "sample":
        lists = rng.random() < 0.3
        n = _log(rng, 2, 64) if lists else rng.choice([V0, _log(rng, 65, V0), _log(rng, 65, V0)])
        return {"op": op, "B": _log(rng, 1, 256), "n": n, "dtype": dtype, "lists": lists, "k": top_k, **how}
    if op == "verify":
        s = _log(rng, 1, 16)
        return {"op": op, "B": _log(rng, 1, max(1, 256 // (s + 1))), "s": s, "n": rng.choice([V0, _log(rng, 1000, V0)]),
                "k": _log(rng, 1, 64), "dtype": dtype, "top_k": top_k, "ragged": rng.random() < 0.5, **how}
    d = rng.choice([8 * _log(rng, 8, 640), _log(rng, 33, 5120)])
    scale = rng.choice([1.0, d ** 0.5])
    V = rng.choice([V0, _log(rng, 1000, V0)])
    if op == "embed":
        return {"op": op, "N": _log(rng, 1, 16384), "V": V, "d": d, "dtype": dtype, "scale": scale}
    V = max(100, min(V, 32003 * 5120 // (d * (2 if dtype == "fp32" else 1))))
    return {"op": op, "N": min(_log(rng, 1, 16384), max(1, 4096 * 5120 // d)), "V": V, "d": d, "dtype": dtype, "scale": scale}


def _model_logits(rows, n, rand, randn):
    """Logits as a language model's rows have them: noise over the vocabulary and some 200 tokens above it that fall
    off by rank, from rows that are sure of a token to rows whose mass lies in the noise. A grammar forbids some tokens
    everywhere, and nearly all of them in a few rows."""
    top = min(n, 200)
    best = 15 + 7 * rand(rows, 1) - (2 + rand(rows, 1)) * torch.log1p(torch.arange(top, device="cuda")) + 0.3 * randn(rows, top)
    edge = torch.arange(top + 1, device="cuda") * n // top
    place = (edge[:-1] + (rand(rows, top) * (edge[1:] - edge[:-1])).long()).minimum(edge[1:] - 1)     # distinct in a row
    place = place.gather(1, rand(rows, top).argsort(1))
    share = torch.where(rand(rows, 1) < 0.05, 0.999, 0.01)
    x = (randn(rows, n) * 2).scatter_(1, place, best).masked_fill_(rand(rows, n) < share, float("-inf"))
    return x.scatter_(1, place[:, :1], best[:, :1])


def _settings(case, rows, rand):
    """temperature, top_k, top_p, min_p: numbers, or tensors of a batch whose requests bring their own."""
    if not case["mixed"]:
        return case["T"], case["k"] if case["op"] == "sample" else case["top_k"], case["p"], case["m"]
    pick = (rand(rows) * len(MIXED)).long().clamp_(max=len(MIXED) - 1)
    T, k, p, m = torch.tensor(MIXED, dtype=torch.float64, device="cuda")[pick].T
    return T.float().contiguous(), k.int().contiguous(), p.float().contiguous(), m.float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op, dt = case["op"], DT[case["dtype"]]
    if op == "sample":
        B, n = case["B"], case["n"]
        if case["lists"]:   # best first, as the draft head returns them; ids distinct in a row
            x = 14 - torch.cumsum(rand(B, n), 1)
            ids = ((torch.arange(n, device="cuda") + rand(B, n)) / n * V0).int().clamp_(max=V0 - 1)
            ids = ids.gather(1, rand(B, n).argsort(1))
        else:
            x, ids = _model_logits(B, n, rand, randn), None
        return {"case": case, "x": x.to(dt), "ids": ids, "u": rand(B), "how": _settings(case, B, rand)}
    if op == "verify":
        B, s, n = case["B"], case["s"], case["n"]
        k = min(case["k"], n)
        x = _model_logits(B * (s + 1), n, rand, randn).view(B, s + 1, n)
        # the drafter's lists: the best of a noisier head, its softmax at the request's temperature, a token drawn from it
        guess, ids = (x[:, :s] + 0.7 * randn(B, s, n)).topk(k, 2)
        T = torch.full((B,), case["T"], device="cuda") if not case["mixed"] else torch.ones(B, device="cuda")
        probs = torch.softmax(guess / T[:, None, None], 2)
        at = (torch.cumsum(probs, 2) <= rand(B, s, 1)).sum(2).clamp_(max=k - 1)
        token = ids.gather(2, at[..., None])[..., 0].int()
        length = (rand(B) * (s + 1)).int().clamp_(max=s) if case["ragged"] else None
        return {"case": case, "x": x.to(dt), "token": token, "u": rand(B, s + 1), "ids": ids.int(), "probs": probs,
                "length": length, "how": _settings(case, B, rand)}
    N, V, d = case["N"], case["V"], case["d"]
    token = (V ** rand(N).double()).int().clamp_(min=1, max=V) - 1    # token r with a probability of about 1 / (r log V)
    if N >= 8:
        token[rand(N) < 0.03] = -1     # padding, and slots that a verification left empty
    if op == "embed":
        return {"case": case, "W": randn(V, d).to(dt), "token": token}
    return {"case": case, "dY": randn(N, d).to(dt), "token": token}


# ------------------------------------------------------------------ plain forms

def _column(v, rows):
    """A setting as a column in 64 bits, of the value that it has in 32."""
    return v.double()[:, None] if isinstance(v, torch.Tensor) else torch.full((rows, 1), v, device="cuda").double()


def _weights_plain(x, how):
    """Weights in 64 bits, 0 for tokens that the settings leave out; rows by columns."""
    rows, n = x.shape
    T, k, p, m = (_column(v, rows) for v in how)
    greedy = T == 0
    T = torch.where(greedy, 1.0, T)
    k = torch.where(greedy, 1.0, torch.where(k == 0, float(n), k))
    x = x.double()
    d = (x - x.amax(1, keepdim=True)) / T
    best, order = x.sort(dim=1, descending=True, stable=True)
    w = torch.exp(d).gather(1, order)
    rank = torch.arange(n, device="cuda")[None]
    w = torch.where(rank < k, w, 0.0)
    before = torch.cumsum(w, 1)
    total = before[:, -1:]
    before = torch.cat([torch.zeros_like(total), before[:, :-1]], 1)
    stay = (rank == 0) | (p >= 1) | (before < p * total)
    stay &= (m <= 0) | (d.gather(1, order) >= torch.log(m))
    return torch.zeros_like(w).scatter_(1, order, torch.where(stay, w, 0.0))


def _draw_plain(w, u):
    c = torch.cumsum(w, 1)
    return (c <= u.double()[:, None] * c[:, -1:]).sum(1).clamp_(max=w.shape[1] - 1)


def _sample_plain(s, case):
    w = _weights_plain(s["x"], s["how"])
    at = _draw_plain(w, s["u"])[:, None]
    q = w / w.sum(1, keepdim=True)
    out = {"token": (at if s["ids"] is None else s["ids"].gather(1, at))[:, 0].int(), "prob": q.gather(1, at)[:, 0].float()}
    if case["lists"]:
        out["probs"] = q.float()
    return out


def _verify_plain(s, case):
    B, n1, n = s["x"].shape
    s1 = n1 - 1
    how = [v.repeat_interleave(n1) if isinstance(v, torch.Tensor) else v for v in s["how"]]
    p = _weights_plain(s["x"].view(B * n1, n), how)
    p = (p / p.sum(1, keepdim=True)).view(B, n1, n)
    token, ids, q = s["token"].long(), s["ids"].long(), s["probs"].double()
    length = torch.full((B,), s1, device="cuda") if s["length"] is None else s["length"].long()
    q_token = torch.where(ids == token[..., None], q, 0.0).sum(2)
    p_token = p[:, :s1].gather(2, token[..., None])[..., 0]
    ok = s["u"][:, :s1].double() * q_token < p_token
    ok &= torch.arange(s1, device="cuda") < length[:, None]
    taken = torch.cumprod(ok.int(), 1).sum(1)
    rows = torch.arange(B, device="cuda")
    last = p[rows, taken]
    at = taken.clamp(max=s1 - 1)
    missed = torch.zeros_like(last).scatter_add_(1, ids[rows, at], q[rows, at])
    rest = (last - missed).clamp_(min=0.0)
    rest = torch.where((taken < length)[:, None] & (rest.sum(1, keepdim=True) > 0), rest, last)
    new = _draw_plain(rest, s["u"][:, s1])
    place = torch.arange(n1, device="cuda")
    out = torch.where(place < taken[:, None], torch.cat([token, token[:, :1]], 1), -1)
    return {"token": torch.where(place == taken[:, None], new[:, None], out).int(), "count": (taken + 1).int()}


def _embed_plain(s, case):
    token = s["token"].long()
    rows = s["W"][token.clamp(min=0)].float() * case["scale"]
    return torch.where((token >= 0)[:, None], rows, 0.0).to(s["W"].dtype)


def _embed_grad_plain(s, case):
    token = s["token"].long()
    rows = torch.where((token >= 0)[:, None], s["dY"].float(), 0.0)
    dW = torch.zeros(case["V"], case["d"], device="cuda").index_add_(0, token.clamp(min=0), rows)
    return (dW * case["scale"]).to(s["dY"].dtype)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"sample": _sample_plain, "verify": _verify_plain, "embed": _embed_plain,
                "embed_grad": _embed_grad_plain}[op](s, case)
    import rank_lm_head_amd as lr
    if op in ("sample", "verify"):
        T, k, p, m = s["how"]
    if op == "sample":
        token, prob, probs = lr.sample(s["x"], s["u"], idx=s["ids"], temperature=T, top_k=k, top_p=p, min_p=m,
                                       want_probs=case["lists"])
        return {"token": token, "prob": prob, "probs": probs} if case["lists"] else {"token": token, "prob": prob}
    if op == "verify":
        token, count = lr.verify(s["x"], s["token"], s["u"], idx=s["ids"], probs=s["probs"], length=s["length"],
                                 temperature=T, top_k=k, top_p=p, min_p=m)
        return {"token": token, "count": count}
    if op == "embed":
        return lr.embed(s["W"], s["token"], scale=case["scale"])
    return lr.embed_grad(s["dY"], s["token"], case["V"], scale=case["scale"])


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        B, n = case["B"], case["n"]
        return {"bytes": B * n * (size + (8 if case["lists"] else 0)) + 12 * B + 16 * B * case["mixed"], "flops": 4 * B * n}
    if case["op"] == "verify":
        B, s, n, k = case["B"], case["s"], case["n"], case["k"]
        rows = B * (s / 2 + 1 if case["ragged"] else s + 1)    # rows of the drafted tokens that there are
        return {"bytes": int(rows * n * size + B * (s * (8 * k + 8) + 12)), "flops": int(4 * rows * n)}
    N, V, d = case["N"], case["V"], case["d"]
    if case["op"] == "embed_grad":
        return {"bytes": (N + V) * d * size + 4 * N, "flops": N * d}
    mass = torch.log1p(1 / torch.arange(1, V + 1, dtype=torch.float64)) / torch.log(torch.tensor(V + 1.0)).item()
    seen = int((1 - (1 - mass) ** N).sum())      # distinct rows read, on average
    return {"bytes": (N + seen) * d * size + 4 * N, "flops": N * d}


# -------------------------------------------------------------- 64-bit results

def _probs_exact(x, how, row):
    """The distribution of one row under its settings, from the definition."""
    T, k, p, m = (float(v[row]) if isinstance(v, torch.Tensor) else float(torch.tensor(v).float()) for v in how)
    x = x.double()
    if T == 0:
        T, k = 1.0, 1
    q = torch.softmax(x / T, 0)
    order = torch.argsort(-x, stable=True)
    if 0 < k < len(x):
        order = order[:int(k)]
    if p < 1:
        some = q[order] / q[order].sum()
        keep = max(1, int((torch.cumsum(some, 0) - some < p).sum()))
        order = order[:keep]
    if m > 0:
        order = order[q[order] >= m * q.max()]
    left = torch.zeros_like(q)
    left[order] = q[order]
    return left / left.sum()


def _pick_exact(q, u):
    """The first place whose sum of probabilities, itself among them, is above u."""
    c = torch.cumsum(q, 0) / q.sum()
    return int(torch.searchsorted(c, u.double().reshape(1), right=True).clamp(max=int(q.nonzero().max())))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        rows = [_probs_exact(x, s["how"], i) for i, x in enumerate(s["x"])]
        at = [_pick_exact(q, s["u"][i]) for i, q in enumerate(rows)]
        token = at if s["ids"] is None else [int(s["ids"][i, j]) for i, j in enumerate(at)]
        out = {"token": torch.tensor(token, dtype=torch.int32), "prob": torch.stack([q[j] for q, j in zip(rows, at)])}
        return {**out, "probs": torch.stack(rows)} if case["lists"] else out
    if case["op"] == "verify":
        out, counts = [], []
        for b in range(case["B"]):
            had = case["s"] if s["length"] is None else int(s["length"][b])
            got = []
            for j in range(had + 1):
                p = _probs_exact(s["x"][b, j], s["how"], b)
                if j < had:
                    x = int(s["token"][b, j])
                    q = torch.zeros_like(p)
                    q.index_add_(0, s["ids"][b, j].long(), s["probs"][b, j].double())
                    if float(s["u"][b, j]) * float(q[x]) < float(p[x]):
                        got.append(x)
                        continue
                    rest = torch.clamp(p - q, min=0)
                    p = rest if float(rest.sum()) > 0 else p
                got.append(_pick_exact(p, s["u"][b, -1]))
                break
            counts.append(len(got))
            out.append(got + [-1] * (case["s"] + 1 - len(got)))
        return {"token": torch.tensor(out, dtype=torch.int32), "count": torch.tensor(counts, dtype=torch.int32)}
    live = s["token"] >= 0
    if case["op"] == "embed":
        y = torch.zeros(case["N"], case["d"], dtype=torch.float64, device="cuda")
        y[live] = torch.index_select(s["W"], 0, s["token"][live]).double() * case["scale"]
        return y
    dW = torch.zeros(case["V"], case["d"], dtype=torch.float64, device="cuda")
    dW.index_put_((s["token"][live].long(),), case["scale"] * s["dY"][live].double(), accumulate=True)
    return dW
