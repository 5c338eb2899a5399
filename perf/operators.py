"""Timed cases of the head's training and beam-search operators.

distill:  the loss of a rank-r student head against a teacher's top logits, and its gradients.
beam:     the selection of the best continuations over beams and vocabulary (or candidate lists).
reorder:  beams' states moved behind their new beams.

`run` computes a case in its plain form (torch operations in 32 bits, in 64 where totals are ranked), or, with `own`
set, through the package.
"""
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
V0 = 151936          # vocabulary of the drafter head
WORK = 4096 * V0 * 128   # N * V * r of the largest distillation step


def listed():
    d = lambda name, **c: {"name": name, "op": "distill", **c}  # noqa: E731
    b = lambda name, **c: {"name": name, "op": "beam", **c}  # noqa: E731
    r = lambda name, **c: {"name": name, "op": "reorder", **c}  # noqa: E731
    return [
        # a training step of the drafter head on one sequence of 4096 positions
        d("distill_step_4096x128", N=4096, V=V0, r=128, k=32, dtype="bf16", train=True, T=1.0),
        # the high-load batch's shape: twice the rank, half the rows, all 64 teacher places
        d("distill_step_2048x256", N=2048, V=V0, r=256, k=64, dtype="bf16", train=True, T=2.0),
        # online distillation from the 64 nodes of one draft tree, rank at its maximum
        d("distill_step_64x512", N=64, V=V0, r=512, k=64, dtype="bf16", train=True, T=1.0),
        # the loss alone, for a held-out set
        d("distill_eval_1000x128", N=1000, V=V0, r=128, k=32, dtype="bf16", train=False, T=1.0),
        # the tiny fp32 head, odd row count
        d("distill_step_tiny_fp32", N=333, V=4096, r=32, k=8, dtype="fp32", train=True, T=1.0),
        # one request, four beams over the full head's dense fp32 logits: latency
        b("beam_dense_1x4", B=1, m=4, n=V0, nb=4, dtype="fp32", lists=False, ended=False),
        # 32 requests, eight beams each, a bf16 head's dense logits
        b("beam_dense_32x8", B=32, m=8, n=V0, nb=8, dtype="bf16", lists=False, ended=True),
        # odd vocabulary, odd beams, more branches than beams
        b("beam_dense_7x5_odd", B=7, m=5, n=32003, nb=10, dtype="fp32", lists=False, ended=True),
        # the draft head's candidate lists of 64 requests with eight beams: a drafter's step
        b("beam_lists_64x8", B=64, m=8, n=32, nb=8, dtype="fp32", lists=True, ended=True),
        # hidden rows of a drafter's beams
        r("reorder_rows_64x8", B=64, m=8, nb=8, states=1, heads=0, len=1, width=5120, dtype="bf16", ragged=False),
        # keys and values of one drafter layer, prompts of different lengths in a cache of 2048
        r("reorder_cache_16x4", B=16, m=4, nb=4, states=2, heads=8, len=2048, width=128, dtype="bf16", ragged=True),
        # short caches of several layers: many small states
        r("reorder_layers_4x5", B=4, m=5, nb=5, states=16, heads=4, len=129, width=64, dtype="bf16", ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["distill", "distill", "beam", "reorder"])
    if op == "distill":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        V = rng.choice([V0, _log(rng, 4096, V0), _log(rng, 4096, V0)])
        r = 8 * _log(rng, 1, 64)
        most = WORK if dtype == "bf16" else WORK // 32
        N = max(1, min(_log(rng, 1, 4096), most // (V * r)))
        return {"op": op, "N": N, "V": V, "r": r, "k": _log(rng, 1, 64), "dtype": dtype,
                "train": rng.random() < 0.75, "T": rng.choice([1.0, 2.0, 0.5])}
    if op == "beam":
        lists = rng.random() < 0.4
        m = _log(rng, 1, 16)
        B = _log(rng, 1, 64)
        n = _log(rng, 4, 64) if lists else max(1000, min(rng.choice([V0, _log(rng, 1000, V0)]), 32 * 8 * V0 // (B * m)))
        return {"op": op, "B": B, "m": m, "n": n, "nb": _log(rng, 1, min(32, m * n)), "dtype": rng.choice(["fp32", "bf16"]),
                "lists": lists, "ended": rng.random() < 0.5}
    B, m, states = _log(rng, 1, 64), _log(rng, 1, 16), _log(rng, 1, 16)
    heads = rng.choice([0, 0, 1, 2, 4, 8])
    width = rng.choice([64, 128]) if heads else 8 * _log(rng, 8, 640)
    room = 16 * 4 * 2 * 8 * 2048 * 128 // (B * m * states * max(1, heads) * width)
    length = max(1, min(_log(rng, 1, 2048), room)) if heads else 1
    return {"op": op, "B": B, "m": m, "nb": max(1, min(16, m + rng.randint(-2, 2))), "states": states, "heads": heads,
            "len": length, "width": width, "dtype": rng.choice(["bf16", "fp32"]), "ragged": heads > 0 and rng.random() < 0.7}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op = case["op"]
    if op == "distill":
        N, V, r, k, dt = case["N"], case["V"], case["r"], case["k"], DT[case["dtype"]]
        P = (randn(V, r) * (2.5 / r ** 0.5)).to(dt)    # scores with a standard deviation of about 2.5
        Z = randn(N, r).to(dt)
        # ids dense towards the frequent end of the vocabulary, distinct in a row where V >= k * k, in no order
        at = (torch.arange(k, device="cuda") + rand(N, k)) / k
        idx = (at * at * V).long().clamp_(max=V - 1)
        idx = idx.gather(1, rand(N, k).argsort(1)).int()
        t = 14 - torch.cumsum(rand(N, k) * 1.5, 1)     # best first, as the full head's top-k returns it
        w = rand(N) / N
        if N >= 8:   # padded rows, and rows with fewer teacher places
            idx[rand(N) < 0.03] = -1
            idx[(rand(N) < 0.1)[:, None] & (torch.arange(k, device="cuda") >= (k + 1) // 2)] = -1
        return {"case": case, "Z": Z, "P": P, "idx": idx, "t": t, "w": w}
    if op == "beam":
        B, m, n, dt = case["B"], case["m"], case["n"], DT[case["dtype"]]
        if case["lists"]:   # best first, as the draft head returns them; ids distinct in a row
            x = 14 - torch.cumsum(rand(B, m, n), 2)
            ids = ((torch.arange(n, device="cuda") + rand(B, m, n)) / n * V0).int().clamp_(max=V0 - 1)
            ids = ids.gather(2, rand(B, m, n).argsort(2))
        else:
            x = randn(B, m, n) * 2.5
            x[rand(B, m, n) < 0.01] = float("-inf")    # tokens that a grammar forbids
            ids = None
        score = -20 * rand(B, m)
        if m > 1:
            score[rand(B) < 0.1, 1:] = float("-inf")   # requests at their first step: one live beam
        ended = (rand(B, m) < 0.1).to(torch.uint8) if case["ended"] else None
        return {"case": case, "x": x.to(dt), "ids": ids, "score": score, "ended": ended}
    B, m, nb, dt = case["B"], case["m"], case["nb"], DT[case["dtype"]]
    inner = (case["heads"], case["len"], case["width"]) if case["heads"] else (case["width"],)
    states = [randn(B, m, *inner).to(dt) for _ in range(case["states"])]
    out = [torch.zeros(B, nb, *inner, dtype=dt, device="cuda") for _ in states]
    parent = (rand(B, nb) * m).int().clamp_(max=m - 1)
    length = (rand(B) * (case["len"] + 1)).int().clamp_(max=case["len"]) if case["ragged"] else None
    return {"case": case, "states": states, "parent": parent, "length": length, "out": out}


# ------------------------------------------------------------------ plain forms

def _distill_plain(s, case):
    T, V = case["T"], case["V"]
    Z, P = s["Z"].float(), s["P"].float()
    have = s["idx"] >= 0
    ids = s["idx"].long().clamp(min=0)
    t = torch.where(have, s["t"] / T, -torch.inf)
    mass = have.any(1)
    e = torch.exp(t - torch.where(mass, t.amax(1), 0.0)[:, None])
    p = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    x = (Z @ P.T) / T
    hi = x.amax(1)
    ex = torch.exp(x - hi[:, None])
    total = ex.sum(1)
    lse = hi + torch.log(total)
    logp = torch.where(p > 0, torch.log(p), 0.0)
    loss = (p * (logp - x.gather(1, ids) + lse[:, None])).sum(1)
    if not case["train"]:
        return {"loss": loss, "lse": lse}
    c = s["w"] / T * mass
    ds = ex * (c / total)[:, None]
    ds.scatter_add_(1, ids, -p * c[:, None])
    return {"loss": loss, "dZ": (ds @ P).to(s["Z"].dtype), "dP": (ds.T @ Z).to(s["P"].dtype)}


def _beam_plain(s, case):
    B, m, n, nb = case["B"], case["m"], case["n"], case["nb"]
    x = s["x"].double()
    hi = x.amax(2, keepdim=True)
    total = x - (hi + torch.log(torch.exp(x - hi).sum(2, keepdim=True))) + s["score"].double()[:, :, None]
    if s["ended"] is not None:
        over = s["ended"].bool()[:, :, None]
        first = torch.arange(n, device=x.device) == 0
        total = torch.where(over, torch.where(first, s["score"].double()[:, :, None], -torch.inf), total)
    total = total.reshape(B, m * n)
    last = total.topk(nb, 1).values[:, -1:]
    above = total > last
    tied = total == last
    taken = above | (tied & (torch.cumsum(tied, 1) <= nb - above.sum(1, keepdim=True)))
    place = torch.where(taken, -torch.arange(m * n, device=x.device, dtype=torch.float64), -torch.inf)
    place = place.topk(nb, 1).indices            # the taken places in ascending order
    best, order = total.gather(1, place).sort(dim=1, descending=True, stable=True)
    place = place.gather(1, order)
    beam = place // n
    token = s["ids"].long().reshape(B, m * n).gather(1, place) if s["ids"] is not None else place % n
    if s["ended"] is not None:
        token = torch.where(s["ended"].bool().gather(1, beam), END, token)
    live = best > -torch.inf
    return {"score": best.float(), "beam": torch.where(live, beam, -1).int(), "token": torch.where(live, token, -1).int()}


END = 2   # the token that ends a beam


def _reorder_plain(s, case):
    rows = torch.arange(case["B"], device="cuda")[:, None]
    parent = s["parent"].long()
    out = [x[rows, parent] for x in s["states"]]
    if s["length"] is not None:
        live = torch.arange(case["len"], device="cuda") < s["length"][:, None]
        live = live[:, None, None, :, None]
        out = [torch.where(live, x, o) for x, o in zip(out, s["out"])]
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"distill": _distill_plain, "beam": _beam_plain, "reorder": _reorder_plain}[op](state, case)
    import rank_lm_head_amd as lr
    if op == "distill":
        s = state
        loss, lse, G = lr.distill(s["Z"], s["P"], s["idx"], s["t"], temperature=case["T"], want_grad=case["train"])
        if not case["train"]:
            return {"loss": loss, "lse": lse}
        dZ, dP = lr.distill_grad(s["Z"], s["P"], s["idx"], s["t"], lse, G, s["w"], temperature=case["T"])
        return {"loss": loss, "dZ": dZ, "dP": dP}
    if op == "beam":
        score, beam, token = lr.beam_select(state["x"], state["score"], case["nb"], idx=state["ids"],
                                            ended=state["ended"], end_id=END)
        return {"score": score, "beam": beam, "token": token}
    return lr.reorder(state["states"], state["parent"], length=state["length"], out=state["out"])


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "distill":
        N, V, r, k = case["N"], case["V"], case["r"], case["k"]
        grads = 2 if case["train"] else 1
        return {"bytes": grads * (N + V) * r * size + N * k * 8 + N * 4 * grads, "flops": 2 * N * V * r * (3 if case["train"] else 1)}
    if case["op"] == "beam":
        B, m, n, nb = case["B"], case["m"], case["n"], case["nb"]
        return {"bytes": B * m * (n * (size + (4 if case["lists"] else 0)) + 4 + case["ended"]) + 12 * B * nb, "flops": 3 * B * m * n}
    share = 0.5 if case["ragged"] else 1.0
    read = case["m"] * (1 - (1 - 1 / case["m"]) ** case["nb"])   # distinct beams read, on average
    cell = case["states"] * max(1, case["heads"]) * case["len"] * case["width"] * size
    return {"bytes": int(case["B"] * (read + case["nb"]) * cell * share), "flops": 0}


# -------------------------------------------------------------- 64-bit results

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "reorder":
        return _reorder_exact(s, case)
    if case["op"] == "beam":
        return _beam_exact(s, case)
    T, N = case["T"], case["N"]
    P = s["P"].double()
    loss = torch.zeros(N, dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    dZ = torch.zeros(N, case["r"], dtype=torch.float64, device="cuda")
    dP = torch.zeros_like(P)
    for a in range(0, N, 512):
        z, ids, t = s["Z"][a:a + 512].double(), s["idx"][a:a + 512].long(), s["t"][a:a + 512].double() / T
        real = ids >= 0
        alive = real.any(1).double()[:, None]
        logp = torch.log_softmax(t.masked_fill(~real, -1e300), 1)
        p = torch.exp(logp) * real
        x = z @ P.T / T
        lse[a:a + 512] = torch.logsumexp(x, 1)
        logq = x - lse[a:a + 512, None]
        loss[a:a + 512] = (p * (logp.masked_fill(~real, 0.0) - logq.gather(1, ids.clamp(min=0)))).sum(1)
        if case["train"]:
            grad = torch.exp(logq) * alive
            n, j = real.nonzero(as_tuple=True)
            grad.index_put_((n, ids[n, j]), -p[n, j], accumulate=True)
            grad *= s["w"][a:a + 512].double()[:, None] / T
            dZ[a:a + 512] = grad @ P
            dP += grad.T @ z
    return {"loss": loss, "dZ": dZ, "dP": dP} if case["train"] else {"loss": loss, "lse": lse}


def _beam_exact(s, case):
    total = torch.log_softmax(s["x"].double(), 2) + s["score"].double()[..., None]
    best = []
    for b in range(case["B"]):
        rows = total[b]
        if s["ended"] is not None:
            gone = s["ended"][b].bool()
            rows = torch.cat([rows[~gone].flatten(), s["score"][b][gone].double(),
                              rows.new_full((case["nb"],), float("-inf"))])
        best.append(rows.flatten().sort(descending=True).values[:case["nb"]])
    return {"score": torch.stack(best), "beam": None, "token": None}


def _reorder_exact(s, case):
    parent = s["parent"].tolist()
    length = s["length"].tolist() if s["length"] is not None else [case["len"]] * case["B"]
    new = []
    for x, o in zip(s["states"], s["out"]):
        o = o.double()
        for b, row in enumerate(parent):
            for j, i in enumerate(row):
                if case["heads"]:
                    o[b, j, :, :length[b]] = x[b, i, :, :length[b]].double()
                else:
                    o[b, j] = x[b, i].double()
        new.append(o)
    return new
