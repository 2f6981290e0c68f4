"""A language model's log-probabilities and the losses that train on them, measured: the
log-probabilities of given tokens (token_logprobs, from logits with gradient or from hidden states and
the output matrix), the clipped policy loss with its KL term (policy_loss) and the preference loss of
pairs of sequences (preference_loss), each with its gradient.

Every case is made from its dict and a seed alone.  With ``own`` false, run() computes the operators
in their plain form (elementary torch operations in float32); with ``own`` true it calls the library.
exact() is the definition in float64, its gradients by differentiation.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _logprobs(name, rows, n, kind, *, ld=0, temperature=1.0, entropy=False, train=False, left_out=0.0):
    return {"name": name, "op": "logprobs", "rows": rows, "n": n, "type": kind, "ld": ld or n, "temperature": temperature,
            "entropy": entropy, "train": train, "left_out": left_out}


def _policy(name, rows, n, kind, *, ld=0, temperature=1.0, clip=(0.2, 0.2), kl=0.0, entropy=0.0, left_out=0.0):
    return {"name": name, "op": "policy", "rows": rows, "n": n, "type": kind, "ld": ld or n, "temperature": temperature,
            "clip_low": clip[0], "clip_high": clip[1], "kl": kl, "entropy": entropy, "left_out": left_out}


def _prefer(name, pairs, length, n, kind, *, ld=0, beta=0.1, smoothing=0.0, margin=0.0, average=False, ref=True, left_out=0.0):
    return {"name": name, "op": "prefer", "pairs": pairs, "length": length, "n": n, "type": kind, "ld": ld or n,
            "beta": beta, "smoothing": smoothing, "margin": margin, "average": average, "ref": ref, "left_out": left_out}


def _head(name, rows, width, n, kind, *, temperature=1.0, entropy=False, left_out=0.0):
    return {"name": name, "op": "head", "rows": rows, "width": width, "n": n, "type": kind, "temperature": temperature,
            "entropy": entropy, "left_out": left_out}


def listed():
    return [
        # One request's last token, scored anew: latency.
        _logprobs("logprobs 1x32768 bf16", 1, 32768, "bf16"),
        # A batch of prompts scored at the sampling temperature, rows padded for alignment, prompts left out.
        _logprobs("logprobs 512x65536 f16 T.7", 512, 65536, "f16", ld=65600, temperature=0.7, left_out=0.2),
        # A training step on log-probabilities and entropies, an odd vocabulary, rows off the 16-byte grid.
        _logprobs("logprobs 1500x128003 f32 train", 1500, 128003, "f32", entropy=True, train=True),
        # Policy steps, loss and gradient: a handful of tokens (latency),
        _policy("policy 16x32768 bf16", 16, 32768, "bf16"),
        # odd sizes with padding tokens, KL, entropy and asymmetric clipping,
        _policy("policy 1001x100001 f16 kl ent", 1001, 100001, "f16", ld=100032, clip=(0.2, 0.28), kl=0.05, entropy=0.01, left_out=0.15),
        # and a large batch of rollouts.
        _policy("policy 4096x131072 bf16 kl", 4096, 131072, "bf16", kl=0.02, temperature=0.8),
        # Preference steps, loss and gradient: a small model's vocabulary and short answers,
        _prefer("prefer 8x64 512 f32", 8, 64, 512, "f32"),
        # a mean over each answer with a margin and no reference, an odd vocabulary, prompts left out,
        _prefer("prefer 5x150 100001 f16 mean", 5, 150, 100001, "f16", beta=2.0, margin=0.5, average=True, ref=False, left_out=0.3),
        # and a large batch against a reference, with smoothed labels.
        _prefer("prefer 8x512 131072 bf16", 8, 512, 131072, "bf16", smoothing=0.1, left_out=0.1),
        # Scoring from hidden states: a few drafted tokens (the output matrix is what counts),
        _head("head 5x1024x32768 bf16", 5, 1024, 32768, "bf16"),
        # odd sizes with entropies,
        _head("head 777x1000x50001 f16 ent", 777, 1000, 50001, "f16", temperature=1.3, entropy=True, left_out=0.1),
        # and the reference model's pass over a batch of rollouts.
        _head("head 4096x2048x131072 bf16", 4096, 2048, 131072, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["logprobs", "policy", "prefer", "head"])
    left_out = rng.choice([0.0, 0.0, 0.1, 0.5])
    temperature = rng.choice([1.0, round(rng.uniform(0.3, 1.5), 3)])
    if op == "head":
        width, n = _log(rng, 16, 4096), _log(rng, 64, 131072)
        rows = _log(rng, 1, max(1, min(4096, (1 << 37) // (width * n))))
        return {"op": op, "rows": rows, "width": width, "n": n, "type": rng.choice(["bf16", "f16"]), "temperature": temperature,
                "entropy": rng.random() < 0.5, "left_out": left_out}
    n = _log(rng, 64, 200000)
    ld = n + rng.choice([0, 0, 1, 5, 64])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op == "prefer":
        pairs = _log(rng, 1, 64)
        length = _log(rng, 1, max(1, min(2048, (1 << 27) // (2 * pairs * n))))
        return {"op": op, "pairs": pairs, "length": length, "n": n, "type": kind, "ld": ld, "beta": round(rng.uniform(0.05, 1.0), 3),
                "smoothing": rng.choice([0.0, 0.1]), "margin": rng.choice([0.0, 0.5]), "average": rng.random() < 0.3,
                "ref": rng.random() < 0.8, "left_out": left_out}
    case = {"op": op, "rows": _log(rng, 1, max(1, min(65536, (1 << 27) // n))), "n": n, "type": kind, "ld": ld,
            "temperature": temperature, "left_out": left_out}
    if op == "logprobs":
        return {**case, "entropy": rng.random() < 0.5, "train": rng.random() < 0.6}
    return {**case, "clip_low": 0.2, "clip_high": rng.choice([0.2, 0.28]), "kl": rng.choice([0.0, 0.05]),
            "entropy": rng.choice([0.0, 0.01])}


def _rows(case):
    return 2 * case["pairs"] * case["length"] if case["op"] == "prefer" else case["rows"]


def _current(logits, tokens, temperature):
    """The tokens' log-probabilities as the inputs are made from them (a few rows at a time)."""
    out = []
    for l, t in zip(logits.split(512), tokens.split(512)):
        x = l.double() / temperature
        out.append(torch.gather(x, 1, t.clamp(min=0)[:, None])[:, 0] - torch.logsumexp(x, 1))
    return torch.cat(out)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dev, dtype, n = "cuda", TYPES[case["type"]], case["n"]
    s = {"case": case}
    if case["op"] == "head":
        # Normed hidden states that lean towards the row of the token that follows.
        rows, width = case["rows"], case["width"]
        stride = -(-width // 8) * 8  # what the matrices are padded to
        weight = torch.randn((n, stride), generator=g, device=dev).mul_(1.5 * width ** -0.5)
        tokens = torch.randint(n, (rows,), generator=g, device=dev)
        hidden = torch.randn((rows, stride), generator=g, device=dev) + weight[tokens] * (2 * torch.rand((rows, 1), generator=g, device=dev))
        s["hidden"], s["weight"] = hidden.to(dtype)[:, :width], weight.to(dtype)[:, :width]
        s["tokens"] = torch.where(torch.rand(rows, generator=g, device=dev) < case["left_out"], -1, tokens)
        return s
    # A row's logits fall with the logarithm of a random rank, at a slope of its own: some rows are
    # nearly certain of their token, others spread over thousands.  The last entries are what
    # vocabularies are padded with: -inf.  Tokens are drawn from the rows, as a model's own are.
    rows = _rows(case)
    logits = torch.empty((rows, case["ld"]), device=dev, dtype=dtype)
    tokens = torch.empty(rows, device=dev, dtype=torch.int64)
    for i in range(0, rows, 2048):
        part = logits[i:i + 2048]
        slope = 1.0 + torch.rand((len(part), 1), generator=g, device=dev)
        v = torch.rand(part.shape, generator=g, device=dev).mul_(n).add_(1).log_().mul_(-slope).add_(12)
        v[:, n - n // 200:] = -math.inf
        part.copy_(v)
        v = part[:, :n].float() - torch.empty((len(part), n), device=dev).exponential_(generator=g).log_()
        tokens[i:i + 2048] = v.argmax(1)
    s["logits"] = logits[:, :n]
    # float16 has no room for gradients of 1e-7: a step in it scales its loss, by a power of two.
    def scale(size):
        return 8.0 * 2.0 ** round(math.log2(size)) if case["type"] == "f16" else 1.0
    temperature = case.get("temperature", 1.0)
    used = torch.rand(rows, generator=g, device=dev) >= case["left_out"]
    if case["op"] == "logprobs":
        s["tokens"] = torch.where(used, tokens, -1)
        if case["train"]:
            s["grad_logprobs"] = scale(1) * torch.randn(rows, generator=g, device=dev)
            s["grad_entropies"] = 0.1 * scale(1) * torch.randn(rows, generator=g, device=dev) if case["entropy"] else None
        return s
    current = _current(s["logits"], tokens, temperature)
    if case["op"] == "policy":
        s["tokens"] = tokens
        # The policy has moved since the rollout; no ratio lies within a part in a hundred of a clip's
        # border, where the loss has a corner and the gradient no value.
        moved = 0.15 * torch.randn(rows, generator=g, device=dev, dtype=torch.float64)
        for border in (math.log(1 - case["clip_low"]), math.log(1 + case["clip_high"])):
            moved = torch.where((moved - border).abs() < 0.01, border + torch.where(moved < border, -0.01, 0.01), moved)
        s["old"] = (current - moved).float()
        s["advantages"] = torch.randn(rows, generator=g, device=dev)
        s["ref"] = (current + 0.1 * torch.randn(rows, generator=g, device=dev)).float() if case["kl"] else None
        used[0] = True
        s["weights"] = scale(rows) * used / used.sum(dtype=torch.float32)  # the mean over what is not padding
        return s
    # Pairs of answers of at most `length` tokens, one behind the other; rows behind the last are padding.
    lengths = torch.randint(max(1, case["length"] // 2), case["length"] + 1, (2 * case["pairs"],), generator=g, device=dev)
    s["offsets"] = torch.cat([torch.zeros(1, device=dev, dtype=torch.int64), lengths.cumsum(0)])
    s["tokens"] = torch.where(used, tokens, -1)
    s["ref"] = (current + 0.2 * torch.randn(rows, generator=g, device=dev)).float() if case["ref"] else None
    s["grad_loss"] = torch.full((), scale(case["pairs"] / case["beta"]), device=dev)
    return s


# ---- the plain forms ---------------------------------------------------------------------------

def _rows_plain(logits, tokens, temperature):
    """x = (l - max) / T, the sums of exp x and of x exp x, and the tokens' x; all float32."""
    l = logits.float()
    x = (l - l.max(1, keepdim=True).values) / temperature
    e = torch.exp(x)
    total = e.sum(1)
    weighted = torch.where(e > 0, x * e, 0.0).sum(1)
    at = torch.gather(x, 1, tokens.clamp(min=0)[:, None])[:, 0]
    return x, e, total, weighted, at


def _gradient_plain(x, e, total, weighted, tokens, g, gh, temperature, live, dtype):
    """Of sum g logprob + gh entropy, by the logits."""
    p = e / total[:, None]
    d = -g[:, None] * p
    if gh is not None:
        d = d - torch.where(p > 0, gh[:, None] * p * (x - (weighted / total)[:, None]), 0.0)
    d = d.scatter_add(1, tokens.clamp(min=0)[:, None], g[:, None])
    return torch.where(live[:, None], d / temperature, 0.0).to(dtype)


def _logprobs_plain(s, logits):
    case, tokens = s["case"], s["tokens"]
    live = tokens >= 0
    x, e, total, weighted, at = _rows_plain(logits, tokens, case["temperature"])
    out = {"logprobs": torch.where(live, at - torch.log(total), 0.0)}
    if case["entropy"]:
        out["entropies"] = torch.where(live, torch.log(total) - weighted / total, 0.0)
    if case.get("train"):
        out["grad_logits"] = _gradient_plain(x, e, total, weighted, tokens, s["grad_logprobs"], s["grad_entropies"],
                                             case["temperature"], live, logits.dtype)
    return out


def _policy_plain(s):
    case, tokens, w, A = s["case"], s["tokens"], s["weights"], s["advantages"]
    live = w != 0
    x, e, total, weighted, at = _rows_plain(s["logits"], tokens, case["temperature"])
    lp = at - torch.log(total)
    ratio = torch.exp(lp - s["old"])
    lo, hi = 1 - case["clip_low"], 1 + case["clip_high"]
    term = -torch.minimum(ratio * A, ratio.clamp(lo, hi) * A)
    clipped = ((A > 0) & (ratio > hi)) | ((A < 0) & (ratio < lo))
    g = torch.where(clipped, 0.0, -A * ratio)
    gh = None
    out = {"logprobs": torch.where(live, lp, 0.0), "clipped": torch.where(live & clipped, w, 0.0).sum()}
    if case["kl"]:
        apart = s["ref"] - lp
        kl = torch.expm1(apart) - apart
        term = term + case["kl"] * kl
        g = g - case["kl"] * torch.expm1(apart)
        out["kl"] = torch.where(live, w * kl, 0.0).sum()
    if case["entropy"]:
        H = torch.log(total) - weighted / total
        term = term - case["entropy"] * H
        gh = -case["entropy"] * w
        out["entropies"] = torch.where(live, H, 0.0)
    out["loss"] = torch.where(live, w * term, 0.0).sum()
    out["grad_logits"] = _gradient_plain(x, e, total, weighted, tokens, w * g, gh, case["temperature"], live, s["logits"].dtype)
    return out


def _sequence_of(offsets, rows):
    """The sequence that each row belongs to, `2 * pairs` where none."""
    return (torch.arange(rows, device=offsets.device)[:, None] >= offsets[None, 1:]).sum(1)


def _prefer_plain(s):
    case, tokens = s["case"], s["tokens"]
    pairs, rows = case["pairs"], len(tokens)
    of = _sequence_of(s["offsets"], rows)
    live = (tokens >= 0) & (of < 2 * pairs)
    x, e, total, weighted, at = _rows_plain(s["logits"], tokens, 1.0)
    lp = torch.where(live, at - torch.log(total), 0.0)
    ratio = torch.where(live, lp - s["ref"], 0.0) if case["ref"] else lp
    zero = torch.zeros(2 * pairs + 1, device=lp.device)
    sums, count = zero.scatter_add(0, of, ratio)[:-1], zero.scatter_add(0, of, live.float())[:-1]
    share = torch.ones_like(count)
    if case["average"]:
        share = 1 / count.clamp(min=1)
    d = case["beta"] * (sums * share)
    margins = d[0::2] - d[1::2] - case["margin"]
    soft = lambda v: torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)  # noqa: E731  log(1 + exp v)
    eps = case["smoothing"]
    out = {"logprobs": lp, "margins": margins, "loss": ((1 - eps) * soft(-margins) + eps * soft(margins)).sum() / pairs}
    slope = (eps / (1 + torch.exp(-margins)) - (1 - eps) / (1 + torch.exp(margins))) * (case["beta"] / pairs) * s["grad_loss"]
    slope = torch.stack([slope, -slope], 1).flatten() * share
    g = torch.where(live, torch.cat([slope, zero[:1]])[of], 0.0)
    out["grad_logits"] = _gradient_plain(x, e, total, weighted, tokens, g, None, 1.0, live, s["logits"].dtype)
    return out


def run(state):
    s, case = state, state["case"]
    if not own:
        if case["op"] == "head":
            return _logprobs_plain(s, s["hidden"].float() @ s["weight"].float().t())
        return {"logprobs": lambda s: _logprobs_plain(s, s["logits"]), "policy": _policy_plain, "prefer": _prefer_plain}[case["op"]](s)
    import streaming_selection_primitive_gb300 as pk
    if case["op"] == "head":
        r = pk.token_logprobs(s["hidden"], s["tokens"], weight=s["weight"], temperature=case["temperature"], entropy=case["entropy"])
        out = {"logprobs": r.logprobs}
        if case["entropy"]:
            out["entropies"] = r.entropies
        return out
    if case["op"] == "logprobs":
        r = pk.token_logprobs(s["logits"], s["tokens"], temperature=case["temperature"], entropy=case["entropy"])
        out = {"logprobs": r.logprobs}
        if case["entropy"]:
            out["entropies"] = r.entropies
        if case["train"]:
            out["grad_logits"] = pk.token_logprobs_backward(s["logits"], s["tokens"], r, grad_logprobs=s["grad_logprobs"],
                                                            grad_entropies=s["grad_entropies"])
        return out
    if case["op"] == "policy":
        r = pk.policy_loss(s["logits"], s["tokens"], s["old"], s["advantages"], ref_logprobs=s["ref"], weights=s["weights"],
                           temperature=case["temperature"], clip_low=case["clip_low"], clip_high=case["clip_high"], kl=case["kl"],
                           entropy=case["entropy"] or None, gradient=True)
        out = {"logprobs": r.logprobs, "clipped": r.clipped}
        if case["kl"]:
            out["kl"] = r.kl
        if case["entropy"]:
            out["entropies"] = r.entropies
        return {**out, "loss": r.loss, "grad_logits": r.grad_logits}
    r = pk.preference_loss(s["logits"], s["tokens"], s["offsets"], ref_logprobs=s["ref"], beta=case["beta"],
                           label_smoothing=case["smoothing"], margin=case["margin"], average=case["average"])
    return {"logprobs": r.logprobs, "margins": r.margins, "loss": r.loss,
            "grad_logits": pk.preference_loss_backward(s["logits"], s["tokens"], r, grad_loss=s["grad_loss"])}


# ---- the definitions in float64 ----------------------------------------------------------------

def _exact_rows(z, tokens, live, temperature):
    """Log-probabilities and entropies of the rows that count, 0 elsewhere."""
    logp = torch.log_softmax(z / temperature, 1)
    lp = torch.gather(logp, 1, tokens.clamp(min=0)[:, None])[:, 0]
    H = -(torch.exp(logp) * logp.masked_fill(logp == -math.inf, 0.0)).sum(1)
    return torch.where(live, lp, 0.0), torch.where(live, H, 0.0)


def _exact_slopes(z, tokens, live, temperature, objective, grad):
    """Value and gradient of an objective of (logprobs, entropies, rows) that is a sum over rows."""
    lps, Hs, ds = [], [], []
    for i in range(0, len(z), 512):
        part = slice(i, i + 512)
        leaf = z[part].double().requires_grad_(grad)
        lp, H = _exact_rows(leaf, tokens[part], live[part], temperature)
        if grad:
            objective(lp, H, part).backward()
            ds.append(leaf.grad)
        lps.append(lp.detach())
        Hs.append(H.detach())
    return torch.cat(lps), torch.cat(Hs), torch.cat(ds) if grad else None


def exact(case, seed):
    s = prepare(case, seed)
    tokens = s["tokens"]
    if case["op"] == "head":
        live, lps, Hs = tokens >= 0, [], []
        for i in range(0, case["rows"], 512):
            z = s["hidden"][i:i + 512].double() @ s["weight"].double().t()
            lp, H = _exact_rows(z, tokens[i:i + 512], live[i:i + 512], case["temperature"])
            lps.append(lp)
            Hs.append(H)
        return {"logprobs": torch.cat(lps), "entropies": torch.cat(Hs)} if case["entropy"] else {"logprobs": torch.cat(lps)}
    z = s["logits"]
    if case["op"] == "logprobs":
        def objective(lp, H, part):
            v = (s["grad_logprobs"][part].double() * lp).sum()
            return v + (s["grad_entropies"][part].double() * H).sum() if case["entropy"] else v
        lp, H, d = _exact_slopes(z, tokens, tokens >= 0, case["temperature"], objective, case["train"])
        out = {"logprobs": lp}
        if case["entropy"]:
            out["entropies"] = H
        if case["train"]:
            out["grad_logits"] = d
        return out
    if case["op"] == "policy":
        w, A, old = s["weights"].double(), s["advantages"].double(), s["old"].double()
        live = s["weights"] != 0
        sums = {"loss": 0.0, "kl": 0.0, "clipped": 0.0}

        def objective(lp, H, part):
            ratio = torch.exp(lp - old[part])
            bounded = ratio.clamp(1 - case["clip_low"], 1 + case["clip_high"])
            term = torch.maximum(-ratio * A[part], -bounded * A[part])
            sums["clipped"] += (w[part] * (live[part] & (bounded * A[part] < ratio * A[part]))).sum()
            if case["kl"]:
                q = s["ref"][part].double() - lp
                k3 = torch.exp(q) - 1 - q
                sums["kl"] += torch.where(live[part], w[part] * k3.detach(), 0.0).sum()
                term = term + case["kl"] * k3
            if case["entropy"]:
                term = term - case["entropy"] * H
            v = torch.where(live[part], w[part] * term, 0.0).sum()
            sums["loss"] += v.detach()
            return v
        lp, H, d = _exact_slopes(z, tokens, live, case["temperature"], objective, True)
        out = {"logprobs": lp, "clipped": sums["clipped"]}
        if case["kl"]:
            out["kl"] = sums["kl"]
        if case["entropy"]:
            out["entropies"] = H
        return {**out, "loss": sums["loss"], "grad_logits": d}
    ends = s["offsets"].tolist()
    live = tokens >= 0
    live[ends[-1]:] = False
    lp, _, _ = _exact_slopes(z, tokens, live, 1.0, None, False)
    leaf = lp.clone().requires_grad_()
    ratio = torch.where(live, leaf - s["ref"].double(), 0.0) if case["ref"] else leaf
    D = []
    for a, b in zip(ends[:-1], ends[1:]):
        total = ratio[a:b].sum()
        D.append(case["beta"] * (total / max(1, int(live[a:b].sum())) if case["average"] else total))
    margins = torch.stack(D[0::2]) - torch.stack(D[1::2]) - case["margin"]
    eps = case["smoothing"]
    loss = -((1 - eps) * torch.nn.functional.logsigmoid(margins) + eps * torch.nn.functional.logsigmoid(-margins)).mean()
    slope, = torch.autograd.grad(loss * s["grad_loss"].double(), leaf)
    _, _, d = _exact_slopes(z, tokens, live, 1.0, lambda lp, H, part: (slope[part] * lp).sum(), True)
    return {"logprobs": lp, "margins": margins.detach(), "loss": loss.detach(), "grad_logits": d}


def work(case):
    n, size = case["n"], SIZE[case["type"]]
    rows = _rows(case)
    live = rows * (1 - case["left_out"])
    if case["op"] == "head":
        return {"bytes": (live + n) * case["width"] * size + rows * (16 if case["entropy"] else 12),
                "flops": 2.0 * live * n * case["width"]}
    if case["op"] == "prefer":  # answers are three quarters of the longest on average, the rest is padding
        live *= 0.75
    grad = case["op"] != "logprobs" or case["train"]
    small = {"logprobs": 12 + (8 if grad else 0), "policy": 28, "prefer": 16}[case["op"]]
    return {"bytes": live * n * size + (rows * n * size if grad else 0) + rows * small,
            "flops": (10.0 if grad else 5.0) * live * n}
