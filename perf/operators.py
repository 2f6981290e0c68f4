"""The selections of a language model, measured: the choice of a token (sample_tokens) and the
choice of each token's experts with counts, balance loss and gradient (route, route_backward).

Every case is made from its dict and a seed alone.  With ``own`` false, run() computes the
operators in their plain form (elementary torch operations in float32); with ``own`` true it calls
the library.  exact() is the definition in float64.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # One request's decoding step, a small vocabulary and the usual filters: latency.
        {"name": "sample 1x32768 bf16 k50 p.9", "op": "sample", "rows": 1, "n": 32768, "type": "bf16", "ld": 32768,
         "temperature": 0.8, "top_k": 50, "top_p": 0.9, "min_p": 0.0, "mask": False, "mixed": False},
        # A few requests of a model with float32 logits, an odd vocabulary, rows off the 16-byte grid.
        {"name": "sample 8x128003 f32 p.95", "op": "sample", "rows": 8, "n": 128003, "type": "f32", "ld": 128003,
         "temperature": 1.0, "top_k": 0, "top_p": 0.95, "min_p": 0.0, "mask": False, "mixed": False},
        # Constrained decoding: a packed mask allows part of the vocabulary; min-p alone.
        {"name": "sample 32x100001 f16 mask", "op": "sample", "rows": 32, "n": 100001, "type": "f16", "ld": 100032,
         "temperature": 1.2, "top_k": 0, "top_p": 1.0, "min_p": 0.05, "mask": True, "mixed": False},
        # A server's batch: every request has its own parameters (greedy, top-k, top-p, min-p, none).
        {"name": "sample 64x131072 bf16 mixed", "op": "sample", "rows": 64, "n": 131072, "type": "bf16", "ld": 131072,
         "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "mask": False, "mixed": True},
        # A large batch under nucleus sampling.
        {"name": "sample 256x131072 bf16 p.9", "op": "sample", "rows": 256, "n": 131072, "type": "bf16", "ld": 131072,
         "temperature": 0.7, "top_k": 0, "top_p": 0.9, "min_p": 0.0, "mask": False, "mixed": False},
        # Rollouts for training: temperature alone, so every token takes part.
        {"name": "sample 512x65536 f32 plain", "op": "sample", "rows": 512, "n": 65536, "type": "f32", "ld": 65536,
         "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "mask": False, "mixed": False},
        # Routing of one decoding step's tokens (no loss): latency.
        {"name": "route 16x128 bf16 k8", "op": "route", "tokens": 16, "experts": 128, "k": 8, "type": "bf16",
         "score": "softmax", "normalize": True, "bias": False, "mask": False, "train": False},
        # Routing of a long prompt, sigmoid scores with a bias that balances the choice (no loss).
        {"name": "route 16384x256 f32 k8 sig", "op": "route", "tokens": 16384, "experts": 256, "k": 8, "type": "f32",
         "score": "sigmoid", "normalize": True, "bias": True, "mask": False, "train": False},
        # Training steps, forward and backward with the balance loss: a small batch of a small model,
        {"name": "balance 4096x64 f32 k2", "op": "route", "tokens": 4096, "experts": 64, "k": 2, "type": "f32",
         "score": "softmax", "normalize": True, "bias": False, "mask": False, "train": True},
        # odd sizes with padding tokens and gates that are the probabilities themselves,
        {"name": "balance 10007x60 bf16 k4 mask", "op": "route", "tokens": 10007, "experts": 60, "k": 4, "type": "bf16",
         "score": "softmax", "normalize": False, "bias": False, "mask": True, "train": True},
        # an ordinary batch,
        {"name": "balance 32768x128 bf16 k8", "op": "route", "tokens": 32768, "experts": 128, "k": 8, "type": "bf16",
         "score": "softmax", "normalize": True, "bias": False, "mask": False, "train": True},
        # and a large one with sigmoid scores.
        {"name": "balance 131072x256 f32 k8 sig", "op": "route", "tokens": 131072, "experts": 256, "k": 8, "type": "f32",
         "score": "sigmoid", "normalize": True, "bias": True, "mask": False, "train": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    if rng.random() < 0.5:
        n = _log(rng, 64, 200000)
        rows = _log(rng, 1, max(1, min(512, 32 * 1024 * 1024 // n)))
        kind = rng.choice(["k", "p", "kp", "m", "none", "mixed", "all"])
        return {"op": "sample", "rows": rows, "n": n, "type": rng.choice(["f32", "bf16", "f16"]),
                "ld": n + rng.choice([0, 0, 1, 5, 64]), "temperature": round(rng.uniform(0.3, 1.5), 3),
                "top_k": _log(rng, 2, 1000) if kind in ("k", "kp", "all") else 0,
                "top_p": round(rng.uniform(0.5, 0.99), 3) if kind in ("p", "kp", "all") else 1.0,
                "min_p": round(rng.uniform(0.01, 0.2), 4) if kind in ("m", "all") else 0.0,
                "mask": rng.random() < 0.25, "mixed": kind == "mixed"}
    experts = _log(rng, 4, 512)
    k = rng.randint(1, min(experts, 16))
    return {"op": "route", "tokens": _log(rng, 1, min(131072, 131072 * 256 // experts)), "experts": experts,
            "k": k, "type": rng.choice(["f32", "bf16", "f16"]),
            "score": rng.choice(["softmax", "sigmoid"]), "normalize": k > 1 and rng.random() < 0.7, "bias": rng.random() < 0.4,
            "mask": rng.random() < 0.4, "train": rng.random() < 0.6}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev, dtype = "cuda", TYPES[case["type"]]
    s = {"case": case}
    if case["op"] == "sample":
        rows, n = case["rows"], case["n"]
        # A row's logits fall with the logarithm of a random rank, at a slope of its own: some rows
        # are nearly certain of their token, others spread over thousands.  The last entries are
        # what vocabularies are padded with: -inf.
        slope = 1.0 + torch.rand((rows, 1), generator=g, device=dev)
        store = torch.rand((rows, case["ld"]), generator=g, device=dev)
        store = -slope * torch.log(store * n + 1) + 0.3 * torch.randn(store.shape, generator=g, device=dev) + 12
        store[:, n - n // 200:] = -math.inf
        s["logits"] = store.to(dtype)[:, :n]
        s["noise"] = torch.empty((rows, n), device=dev).exponential_(generator=g)
        if case["mask"]:
            words = -(-n // 32)
            s["mask"] = torch.randint(-(1 << 31), 1 << 31, (rows, words), generator=g, device=dev).to(torch.int32)
            if rows > 1:
                s["mask"][rows // 2] = 0  # a request whose grammar allows nothing
        else:
            s["mask"] = None
        s["temperature"] = torch.full((rows,), case["temperature"], device=dev)
        s["top_k"] = torch.full((rows,), case["top_k"], device=dev, dtype=torch.int32)
        s["top_p"] = torch.full((rows,), case["top_p"], device=dev)
        s["min_p"] = torch.full((rows,), case["min_p"], device=dev)
        if case["mixed"]:
            r = torch.arange(rows, device=dev) % 8
            s["temperature"] = torch.where(r == 0, 0.0, 0.6 + 0.1 * r.float())
            s["top_k"] = torch.where((r == 1) | (r == 2), 40, 0).to(torch.int32)
            s["top_p"] = torch.where((r == 2) | (r == 3) | (r == 4) | (r == 6), 0.9, 1.0)
            s["min_p"] = torch.where((r == 5) | (r == 6), 0.05, 0.0)
        return s
    tokens, experts = case["tokens"], case["experts"]
    z = 1.5 * torch.randn((tokens, experts), generator=g, device=dev)
    z += 0.5 * torch.randn((1, experts), generator=g, device=dev)  # experts differ in how often they are wanted
    s["logits"] = z.to(dtype)
    s["bias"] = 0.3 * torch.randn(experts, generator=g, device=dev) if case["bias"] else None
    s["mask"] = torch.rand(tokens, generator=g, device=dev) < 0.9 if case["mask"] else None
    if case["mask"]:
        s["mask"][0] = True  # the rest: one token in ten is padding
    if case["train"]:  # of a loss summed over the tokens
        s["grad_gates"] = torch.randn((tokens, case["k"]), generator=g, device=dev)
        s["grad_loss"] = torch.full((), 0.01 * tokens, device=dev)
    return s


# ---- the plain forms ---------------------------------------------------------------------------

def _sample_plain(s):
    l = s["logits"].float() + 0.0
    rows, n = l.shape
    if s["mask"] is not None:
        bit = torch.arange(n, device=l.device)
        allowed = (s["mask"][:, bit // 32] >> (bit % 32)) & 1 == 1
    else:
        allowed = torch.ones_like(l, dtype=torch.bool)
    T, p, a = s["temperature"][:, None], s["top_p"][:, None], s["min_p"][:, None]
    bad = (torch.isnan(l) & allowed).any(1) | ~(T[:, 0] >= 0) | torch.isnan(p[:, 0]) | torch.isnan(a[:, 0])
    l = torch.where(allowed & ~torch.isnan(l), l, -math.inf)
    l, idx = torch.sort(l, dim=1, descending=True, stable=True)
    m = l[:, :1]
    x = torch.where(l == m, 0.0, (l - m) / T)
    rank = torch.arange(n, device=l.device)[None]
    k = torch.where(s["top_k"] > 0, s["top_k"], n)[:, None]
    k = torch.where(T == 0, 1, k)
    keep = (rank < k) & (l > -math.inf) & (x > -math.inf)
    w = torch.where(keep, torch.exp(x), 0.0)
    mass = torch.cumsum(w, 1)
    before = torch.cat([torch.zeros_like(mass[:, :1]), mass[:, :-1]], 1)
    keep &= (before < p * w.sum(1, keepdim=True)) | (p >= 1) | (rank == 0)
    keep &= w >= a.clamp(max=1)
    w = torch.where(keep, w, 0.0)
    score = torch.where(keep, x - torch.log(torch.gather(s["noise"], 1, idx)), -math.inf)
    best = score.max(1, keepdim=True).values
    token = torch.where(keep & (score == best), idx, n).min(1, keepdim=True).values
    x_token = torch.where(idx == token, x, -math.inf).max(1).values
    none, token = ~keep.any(1), token[:, 0]
    logprob = x_token - torch.log(w.sum(1))
    logprob = torch.where(none, -math.inf, logprob)
    return {"tokens": torch.where(bad | none, -1, token), "logprobs": torch.where(bad, math.nan, logprob)}


def _route_plain(s):
    case = s["case"]
    z = s["logits"].float() + 0.0
    tokens, E, k = case["tokens"], case["experts"], case["k"]
    c = z if s["bias"] is None else z + s["bias"]
    c = torch.where(torch.isnan(c), -math.inf, c)
    if s["mask"] is not None:
        c = torch.where(s["mask"][:, None], c, -math.inf)
    c, order = torch.sort(c, dim=1, descending=True, stable=True)
    ok, order = c[:, :k] > -math.inf, order[:, :k]
    chosen = torch.where(ok, order, -1)
    sigmoid = case["score"] == "sigmoid"
    y = torch.minimum(z, torch.zeros_like(z)) - torch.log1p(torch.exp(-z.abs())) if sigmoid else z
    m = y.max(1, keepdim=True).values
    e = torch.where(y == m, 1.0, torch.exp(y - m))
    prob = e / e.sum(1, keepdim=True)
    if case["normalize"]:
        yc = torch.where(ok, torch.gather(y, 1, order), -math.inf)
        ec = torch.where(ok, torch.exp(yc - yc.max(1, keepdim=True).values), 0.0)
        gates = torch.where(ok, ec / ec.sum(1, keepdim=True), 0.0)
    else:
        gates = torch.where(ok, torch.gather(torch.exp(y) if sigmoid else prob, 1, order), 0.0)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=z.device).scatter_add_(
        0, torch.where(ok, order, E).reshape(-1), torch.ones_like(order).reshape(-1))[:E]
    out = {"gates": gates, "experts": chosen, "counts": counts}
    if not case["train"]:
        return out
    N = counts.sum().float().clamp(min=1)
    filled = ok.sum(1, keepdim=True).float()
    live = filled > 0
    share = counts.float() / N
    P = torch.where(live, prob * filled, 0.0).sum(0) / N
    out["loss"] = E * (share * P).sum()
    dg = s["grad_gates"]
    a = s["grad_loss"] * E * share[None] * filled / N
    dy = prob * (a - (prob * a).sum(1, keepdim=True))
    if case["normalize"]:
        d = gates * (dg - (gates * dg).sum(1, keepdim=True))
    elif sigmoid:
        d = gates * dg
    else:
        dy = dy - prob * (gates * dg).sum(1, keepdim=True)
        d = gates * dg
    dy = dy.scatter_add(1, order, torch.where(ok, d, 0.0))
    dz = dy / (1 + torch.exp(z)) if sigmoid else dy
    out["grad_logits"] = torch.where(live, dz, 0.0).to(s["logits"].dtype)
    return out


def run(state):
    case = state["case"]
    if not own:
        return _sample_plain(state) if case["op"] == "sample" else _route_plain(state)
    import streaming_selection_primitive_gb300 as pk
    if case["op"] == "sample":
        tokens, logprobs = pk.sample_tokens(state["logits"], state["noise"], temperature=state["temperature"],
                                            top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"],
                                            mask=state["mask"])
        return {"tokens": tokens, "logprobs": logprobs}
    r = pk.route(state["logits"], case["k"], score=case["score"], normalize=case["normalize"], bias=state["bias"],
                 mask=state["mask"], balance=case["train"])
    out = {"gates": r.gates, "experts": r.experts, "counts": r.counts}
    if case["train"]:
        out["loss"] = r.loss
        out["grad_logits"] = pk.route_backward(state["logits"], r, grad_gates=state["grad_gates"],
                                               grad_loss=state["grad_loss"])
    return out


# ---- the definitions in float64 ----------------------------------------------------------------

def _exact_row(l, q, allowed, T, k, p, a):
    """One row's token and log-probability, from sets: numpy float64."""
    if not T >= 0 or np.isnan(p) or np.isnan(a) or np.isnan(l[allowed]).any():
        return -1, np.nan
    live = np.flatnonzero(allowed & (l > -np.inf))
    if not live.size:
        return -1, -np.inf
    v = l[live]
    order = live[np.argsort(-v, kind="stable")]
    if T == 0:
        return int(order[0]), 0.0
    x = (l[order] - l[order[0]]) / T
    if k > 0:
        order, x = order[:k], x[:k]
    w = np.exp(x)
    if p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        keep = max(1, int(np.searchsorted(before, p * w.sum(), side="left")))
        order, x, w = order[:keep], x[:keep], w[:keep]
    keep = w >= min(a, 1.0)
    order, x, w = order[keep], x[keep], w[keep]
    j = int(np.argmax(x - np.log(q[order])))
    return int(order[j]), float(x[j] - np.log(w.sum()))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        if case["rows"] * case["n"] > 1 << 26:
            return None
        l, q = s["logits"].double().cpu().numpy(), s["noise"].double().cpu().numpy()
        rows, n = l.shape
        par = [s[name].double().cpu().numpy() for name in ("temperature", "top_k", "top_p", "min_p")]
        if s["mask"] is None:
            bits = np.ones((rows, n), bool)
        else:
            words = s["mask"].cpu().numpy().view(np.uint8)
            bits = np.unpackbits(words.reshape(rows, -1), axis=1, bitorder="little")[:, :n].astype(bool)
        got = [_exact_row(l[r], q[r], bits[r], float(par[0][r]), int(par[1][r]), float(par[2][r]), float(par[3][r]))
               for r in range(rows)]
        return {"tokens": None, "logprobs": np.array([v for _, v in got], np.float64)}
    z = s["logits"].double().requires_grad_(case["train"])
    E, k = case["experts"], case["k"]
    with torch.no_grad():  # the choice is made on float32 sums: z + bias as the operator defines it
        c = s["logits"].float() if s["bias"] is None else s["logits"].float() + s["bias"]
        order = torch.argsort(c.double(), dim=1, descending=True, stable=True)[:, :k]
        used = torch.ones(case["tokens"], 1, dtype=torch.bool, device=c.device) if s["mask"] is None else s["mask"][:, None]
        hot = torch.zeros_like(c, dtype=torch.float64).scatter_(1, order, 1.0) * used
    scores = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
    picked = torch.gather(scores, 1, order)
    gates = picked / picked.sum(1, keepdim=True) if case["normalize"] else picked
    gates = gates * used
    out = {"gates": gates.detach(), "experts": None, "counts": None}
    if case["train"]:
        prob = scores / scores.sum(1, keepdim=True)
        per = hot.sum(0)
        loss = E * ((per / per.sum().clamp(min=1)) * (prob * hot.sum(1, keepdim=True)).sum(0) / per.sum().clamp(min=1)).sum()
        (s["grad_loss"].double() * loss + (s["grad_gates"].double() * gates).sum()).backward()
        out["loss"], out["grad_logits"] = loss.detach(), z.grad
    return out


def work(case):
    if case["op"] == "sample":
        rows, n = case["rows"], case["n"]
        # The noise is needed only where a token is kept: everywhere without a filter, nearly nowhere with one.
        free = case["top_k"] <= 0 and case["top_p"] >= 1 and case["min_p"] <= 0
        noise = rows / 8 if case["mixed"] else rows if free else 0
        if case["mask"]:
            noise /= 2
        return {"bytes": rows * n * SIZE[case["type"]] + noise * n * 4 + (rows * n / 8 if case["mask"] else 0) + rows * 28,
                "flops": 4.0 * rows * n}
    t, E, k = case["tokens"], case["experts"], case["k"]
    out = t * k * 12 + E * 8
    b = t * E * SIZE[case["type"]] + out + (t if case["mask"] else 0) + (E * 4 if case["bias"] else 0)
    if case["train"]:
        b += t * E * SIZE[case["type"]] + t * k * 4 + 8
    return {"bytes": b, "flops": (16.0 if case["train"] else 6.0) * t * E}
