"""The row-softmax operators of language models, as cases to measure: log probabilities of
given tokens, the same straight from states and an output embedding, routing to experts, and
the Sinkhorn bias that balances the experts' load.

Each case runs in one of two forms. The plain form is elementary torch operations in 32 bits
(64 where a selection lies next to a border); the other form makes the calls that a user makes
of ``streaming_sinkhorn_b200``.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---- cases ----------------------------------------------------------------------------------

def listed():
    return [
        # one decoding step that reports the sampled token and 20 alternatives (latency)
        _tokens("tokens_decode", 1, 128000, "bf16", top=20, masked=0.0, train=False),
        # scoring a ragged batch of prompts in float32, a vocabulary of odd size, some words banned
        _tokens("tokens_score_odd", 1531, 50257, "fp32", top=5, masked=0.02, train=False),
        # a training step of a policy: log probabilities, an entropy bonus, and their gradient
        _tokens("tokens_train", 4096, 65536, "bf16", top=0, masked=0.0, train=True),
        # a few sequences decoded together, straight from the states (the embedding is read once)
        _linear("linear_decode", 4, 128000, 4096, train=False),
        # scoring a prompt with a vocabulary of odd size
        _linear("linear_score_odd", 1531, 50257, 1024, train=False),
        # a training step: loss, entropy, and the gradients of the states and the embedding
        _linear("linear_train", 4096, 65536, 2048, train=True),
        # the router of one decoding step of eight sequences (latency)
        _route("route_decode", 8, 256, 8, "fp32", "sigmoid", True, 8, 4, True, train=False),
        # the router of a prompt, softmax scores taken as they are
        _route("route_prompt", 16384, 64, 6, "bf16", "softmax", False, 1, 1, False, train=False),
        # a training step of a router with a balancing bias and groups: weights, load, gradient
        _route("route_train", 32768, 256, 8, "fp32", "sigmoid", True, 8, 4, True, train=True),
        # balancing a small micro-batch
        _balance("balance_small", 512, 16, "fp32", "softmax", 0.1, 8),
        # balancing a micro-batch of a mid-sized router
        _balance("balance_mid", 8191, 64, "bf16", "sigmoid", 0.05, 10),
        # balancing a large batch: the score matrix no longer fits on chip
        _balance("balance_large", 65536, 256, "fp32", "sigmoid", 0.05, 20),
    ]


def _tokens(name, rows, vocab, dtype, top, masked, train):
    return {"name": name, "op": "tokens", "rows": rows, "vocab": vocab, "dtype": dtype,
            "top": top, "masked": masked, "train": train}


def _linear(name, rows, vocab, dim, train):
    return {"name": name, "op": "linear", "rows": rows, "vocab": vocab, "dim": dim,
            "train": train}


def _route(name, rows, experts, k, dtype, score, bias, groups, top_groups, renormalize, train):
    return {"name": name, "op": "route", "rows": rows, "experts": experts, "k": k,
            "dtype": dtype, "score": score, "bias": bias, "groups": groups,
            "top_groups": top_groups, "renormalize": renormalize, "train": train}


def _balance(name, rows, experts, dtype, score, eps, n_iters):
    return {"name": name, "op": "balance", "rows": rows, "experts": experts, "dtype": dtype,
            "score": score, "eps": eps, "n_iters": n_iters}


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tokens", "linear", "route", "balance"])
    if op == "tokens":
        vocab = _log_int(rng, 1000, 262144)
        rows = _log_int(rng, 1, max(1, min(16384, (1 << 28) // vocab)))
        train = rng.random() < 0.5
        c = _tokens("", rows, vocab, rng.choice(["bf16", "fp16", "fp32"]),
                    0 if train else rng.choice([0, 1, 5, 8, 20]), rng.choice([0.0, 0.02]), train)
        if c["dtype"] == "fp32":
            c["rows"] = max(1, c["rows"] // 2)
    elif op == "linear":
        dim = 8 * _log_int(rng, 8, 512)
        vocab = _log_int(rng, 1000, min(262144, (1 << 29) // dim))
        rows = _log_int(rng, 1, max(1, min(8192, (1 << 38) // (vocab * dim), (1 << 28) // vocab)))
        c = _linear("", rows, vocab, dim, rng.random() < 0.5)
    elif op == "route":
        groups, per = rng.choice([(1, 8), (1, 60), (1, 64), (1, 160), (1, 384), (4, 16), (8, 20),
                                  (8, 32)])
        experts = groups * per
        top_groups = 1 if groups == 1 else rng.choice([2, groups // 2])
        k = rng.choice([1, 2, 4, 6, 8])
        rows = _log_int(rng, 1, (1 << 23) // experts)
        # (the weight of a single expert renormalises to 1: nothing to compute)
        c = _route("", rows, experts, k, rng.choice(["bf16", "fp32"]),
                   rng.choice(["softmax", "sigmoid"]), rng.random() < 0.6, groups, top_groups,
                   k > 1 and rng.random() < 0.6, rng.random() < 0.5)
    else:
        experts = rng.choice([8, 16, 60, 64, 128, 160, 256])
        rows = _log_int(rng, max(64, 4 * experts), (1 << 24) // experts)
        score = rng.choice(["softmax", "sigmoid"])
        # eps at the scale of the scores: softmax scores are about 1 / experts
        eps = rng.choice([0.05, 0.1, 0.2]) if score == "sigmoid" else rng.choice([0.5, 1, 2]) / experts
        c = _balance("", rows, experts, rng.choice(["bf16", "fp32"]), score, eps,
                     rng.randint(3, 20))
    del c["name"]
    return c


# ---- inputs ---------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows = case["rows"]
    s = {"case": case}
    if case["op"] in ("tokens", "linear"):
        vocab = case["vocab"]
        ids = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        if rows >= 16:  # the prompt's and the padding's tokens are not asked about
            ids = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.1, -100, ids)
        s["ids"] = ids
        if case["train"]:
            # an advantage for each token, and an entropy bonus, as shares of the batch's mean
            s["g_logprob"] = -normal(rows) / rows
            s["g_entropy"] = torch.full((rows,), -0.01 / rows, device="cuda")
    if case["op"] == "tokens":
        z = 2.5 * normal(rows, vocab)
        likely = torch.rand(rows, generator=g, device="cuda") < 0.7
        z[torch.arange(rows, device="cuda"), ids.clamp(min=0)] += 8.0 * likely
        if case["masked"]:
            z.masked_fill_(torch.rand(rows, vocab, generator=g, device="cuda") < case["masked"],
                           -math.inf)
        s["logits"] = z.to(DTYPES[case["dtype"]])
    elif case["op"] == "linear":
        dim = case["dim"]
        s["w"] = (normal(vocab, dim) * (1.5 / math.sqrt(dim))).to(torch.bfloat16)
        s["x"] = (normal(rows, dim) + 0.0).to(torch.bfloat16)
    elif case["op"] == "route":
        e = case["experts"]
        favour = 0.7 * normal(e)  # some experts are liked by all tokens
        s["logits"] = (normal(rows, e) + favour).to(DTYPES[case["dtype"]])
        s["bias"] = -0.1 * favour + 0.01 * normal(e) if case["bias"] else None
        if case["train"]:
            s["g_weights"] = normal(rows, case["k"])
    else:
        e = case["experts"]
        s["logits"] = (normal(rows, e) + 0.7 * normal(e)).to(DTYPES[case["dtype"]])
    if case.get("train"):
        for name in ("logits", "x", "w"):
            if name in s:
                s[name].requires_grad_(True)
    return s


# ---- the operators ----------------------------------------------------------------------------

def run(state):
    return (_own_forms if own else _plain_forms)[state["case"]["op"]](state)


def _own_tokens(s):
    import streaming_sinkhorn_b200 as fs
    c = s["case"]
    out = fs.token_logprobs(s["logits"], s["ids"], top=c["top"])
    r = {"logprobs": out.logprobs, "entropy": out.entropy}
    if c["top"]:
        r["top_logprobs"], r["top_ids"] = out.top_logprobs, out.top_ids
    if c["train"]:
        r["grad"], = torch.autograd.grad((out.logprobs, out.entropy), (s["logits"],),
                                         (s["g_logprob"], s["g_entropy"]))
    return r


def _own_linear(s):
    import streaming_sinkhorn_b200 as fs
    out = fs.linear_logprobs(s["x"], s["w"], s["ids"])
    r = {"logprobs": out.logprobs, "entropy": out.entropy}
    if s["case"]["train"]:
        r["grad_x"], r["grad_w"] = torch.autograd.grad(
            (out.logprobs, out.entropy), (s["x"], s["w"]), (s["g_logprob"], s["g_entropy"]))
    return r


def _own_route(s):
    import streaming_sinkhorn_b200 as fs
    c = s["case"]
    out = fs.route(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                   top_groups=c["top_groups"], renormalize=c["renormalize"], load=c["train"])
    r = {"weights": out.weights, "ids": out.ids}
    if c["train"]:
        r["load"] = out.load
        r["grad"], = torch.autograd.grad(out.weights, s["logits"], s["g_weights"])
    return r


def _own_balance(s):
    import streaming_sinkhorn_b200 as fs
    c = s["case"]
    f, g = fs.balance(s["logits"], score=c["score"], eps=c["eps"], n_iters=c["n_iters"])
    return {"f": f, "g": g}


_own_forms = {"tokens": _own_tokens, "linear": _own_linear, "route": _own_route,
              "balance": _own_balance}


# The plain forms: 32 bits, elementary operations, one rounding at the end.

def _row_softmax(z):
    """(log-sum-exp, probabilities, entropy) of each row; a masked entry has probability 0."""
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    p = e / total
    lse = top + torch.log(total)
    entropy = lse[:, 0] - (p * torch.where(p > 0, z, 0.0)).sum(1)
    return lse, p, entropy


def _score_grad(z, lse, p, entropy, ids, s):
    """The gradient of the scores from those of the log probabilities and the entropies."""
    asked = (ids >= 0)[:, None]
    gl, ge = s["g_logprob"][:, None], s["g_entropy"][:, None]
    logp = torch.where(p > 0, z - lse, 0.0)
    d = p * (-gl - ge * (logp + entropy[:, None]))
    d.scatter_add_(1, ids.clamp(min=0)[:, None], gl)
    return torch.where(asked, d, 0.0)


def _plain_tokens(s):
    c, ids = s["case"], s["ids"]
    z = s["logits"].detach().float()
    asked = ids >= 0
    lse, p, entropy = _row_softmax(z)
    given = z.gather(1, ids.clamp(min=0)[:, None])[:, 0]
    r = {"logprobs": torch.where(asked, given - lse[:, 0], 0.0),
         "entropy": torch.where(asked, entropy, 0.0)}
    if c["top"]:
        # the largest first, ties by the lowest index: one whole number that orders both
        bits = (z + 0.0).view(torch.int32).long()
        bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        key = bits * (1 << 20) - torch.arange(c["vocab"], device=z.device)
        at = key.topk(c["top"], dim=1).indices
        r["top_logprobs"] = torch.where(asked[:, None], z.gather(1, at) - lse, -math.inf)
        r["top_ids"] = torch.where(asked[:, None], at, -1).int()
    if c["train"]:
        r["grad"] = _score_grad(z, lse, p, entropy, ids, s).to(s["logits"].dtype)
    return r


def _plain_linear(s):
    ids = s["ids"]
    x, w = s["x"].detach().float(), s["w"].detach().float()
    z = x @ w.t()
    asked = ids >= 0
    lse, p, entropy = _row_softmax(z)
    given = z.gather(1, ids.clamp(min=0)[:, None])[:, 0]
    r = {"logprobs": torch.where(asked, given - lse[:, 0], 0.0),
         "entropy": torch.where(asked, entropy, 0.0)}
    if s["case"]["train"]:
        d = _score_grad(z, lse, p, entropy, ids, s)
        r["grad_x"] = (d @ w).to(torch.bfloat16)
        r["grad_w"] = (d.t() @ x).to(torch.bfloat16)
    return r


def _scores(z, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    e = torch.exp(z - z.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    c = s["case"]
    z = s["logits"].detach().double()  # 64 bits: which experts are picked is decided at borders
    rows, experts = z.shape
    score = _scores(z, c["score"])
    by = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        groups, per = c["groups"], experts // c["groups"]
        best = by.view(rows, groups, per).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        is_kept = torch.zeros(rows, groups, dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        by = torch.where(is_kept.repeat_interleave(per, 1), by, -math.inf)
    ids = by.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    chosen = score.gather(1, ids)
    total = chosen.sum(1, keepdim=True) if c["renormalize"] else torch.ones_like(chosen[:, :1])
    r = {"weights": (chosen / total).float(), "ids": ids.int()}
    if c["train"]:
        r["load"] = torch.zeros(experts, dtype=torch.int32, device=z.device).scatter_add_(
            0, ids.reshape(-1), torch.ones(ids.numel(), dtype=torch.int32, device=z.device))
        gw = s["g_weights"].double()
        if c["renormalize"]:
            ds = (gw - (gw * chosen / total).sum(1, keepdim=True)) / total
        else:
            ds = gw
        if c["score"] == "sigmoid":
            d = torch.zeros_like(z).scatter_(1, ids, ds * chosen * (1.0 - chosen))
        else:
            d = -score * (ds * chosen).sum(1, keepdim=True)
            d.scatter_add_(1, ids, ds * chosen)
        r["grad"] = d.to(s["logits"].dtype)
    return r


def _plain_balance(s):
    c = s["case"]
    score = _scores(s["logits"].float(), c["score"]) / c["eps"]
    g = torch.zeros(c["experts"], device=score.device)
    for _ in range(c["n_iters"]):
        # means in place of sums with the weights' logarithms, which would cancel
        t = score + g
        top = t.amax(1, keepdim=True)
        f = -(top + torch.log(torch.exp(t - top).mean(1, keepdim=True)))
        t = score + f
        top = t.amax(0)
        g = -(top + torch.log(torch.exp(t - top).mean(0)))
    return {"f": c["eps"] * f[:, 0], "g": c["eps"] * g}


_plain_forms = {"tokens": _plain_tokens, "linear": _plain_linear, "route": _plain_route,
                "balance": _plain_balance}


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    rows = case["rows"]
    if case["op"] == "tokens":
        n = rows * case["vocab"]
        b = n * SIZE[case["dtype"]] + rows * (16 + 8 * case["top"])
        return {"bytes": b + (n * SIZE[case["dtype"]] + 8 * rows if case["train"] else 0),
                "flops": n * (12 if case["train"] else 6)}
    if case["op"] == "linear":
        n, d, v = rows, case["dim"], case["vocab"]
        b = 2 * (n + v) * d + 16 * n
        return {"bytes": b + (2 * (n + v) * d + 8 * n if case["train"] else 0),
                "flops": 2 * n * v * d * (3 if case["train"] else 1)}
    n = rows * case["experts"]
    if case["op"] == "route":
        b = n * SIZE[case["dtype"]] + 8 * rows * case["k"] + 4 * case["experts"]
        return {"bytes": b + (n * SIZE[case["dtype"]] + 4 * rows * case["k"] if case["train"] else 0),
                "flops": 8 * n}
    return {"bytes": n * SIZE[case["dtype"]] + 4 * (rows + case["experts"]),
            "flops": 5 * n * case["n_iters"]}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"tokens": _exact_tokens, "linear": _exact_linear, "route": _exact_route,
            "balance": _exact_balance}[case["op"]](case, s)


def _exact_rows(z, ids, s, lo, hi, train):
    """(log probabilities, entropy, gradient of the scores) of rows lo..hi, z in 64 bits."""
    logp = torch.log_softmax(z, dim=1)
    p = torch.exp(logp)
    h = torch.special.entr(p).sum(1)
    i = ids[lo:hi]
    known = i >= 0
    r = torch.arange(hi - lo, device=z.device)
    lp = torch.where(known, logp[r, i.clamp(min=0)], 0.0)
    d = None
    if train:
        gl, ge = s["g_logprob"][lo:hi].double(), s["g_entropy"][lo:hi].double()
        hot = torch.zeros_like(p)
        hot[r, i.clamp(min=0)] = 1.0
        # d logp = hot - p, d H = -p (log p + H)
        d = gl[:, None] * (hot - p) + ge[:, None] * (torch.special.entr(p) - p * h[:, None])
        d[~known] = 0.0
    return lp, torch.where(known, h, 0.0), d, logp, known


def _exact_tokens(case, s):
    rows, step = case["rows"], max(1, (1 << 26) // case["vocab"])
    out = {"logprobs": [], "entropy": [], "top_logprobs": [], "grad": []}
    for lo in range(0, rows, step):
        hi = min(rows, lo + step)
        z = s["logits"].detach()[lo:hi].double()
        lp, h, d, logp, known = _exact_rows(z, s["ids"], s, lo, hi, case["train"])
        out["logprobs"].append(lp)
        out["entropy"].append(h)
        if case["top"]:
            best = logp.topk(case["top"], dim=1).values
            best[~known] = -math.inf
            out["top_logprobs"].append(best)
        if case["train"]:
            out["grad"].append(d)
    r = {k: torch.cat(v) for k, v in out.items() if v}
    if case["top"]:
        r["top_ids"] = None
    return r


def _exact_linear(case, s):
    rows, step = case["rows"], max(1, (1 << 26) // case["vocab"])
    x, w = s["x"].detach().double(), s["w"].detach().double()
    lps, hs, gx, gw = [], [], [], torch.zeros_like(w) if case["train"] else None
    for lo in range(0, rows, step):
        hi = min(rows, lo + step)
        lp, h, d, _, _ = _exact_rows(x[lo:hi] @ w.t(), s["ids"], s, lo, hi, case["train"])
        lps.append(lp)
        hs.append(h)
        if case["train"]:
            gx.append(d @ w)
            gw += d.t() @ x[lo:hi]
    r = {"logprobs": torch.cat(lps), "entropy": torch.cat(hs)}
    if case["train"]:
        r["grad_x"], r["grad_w"] = torch.cat(gx), gw
    return r


def _exact_route(case, s):
    z = s["logits"].detach().double().requires_grad_(True)
    prob = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, dim=1)
    by = prob.detach().clone()
    if s["bias"] is not None:
        by += s["bias"].double()
    rows = torch.arange(z.shape[0], device=z.device)
    if case["groups"] > 1:
        parts = by.view(z.shape[0], case["groups"], -1)
        left = parts.topk(2, dim=2).values.sum(2)
        keep = torch.zeros_like(left, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            best = left.argmax(1)
            keep[rows, best] = True
            left[rows, best] = -math.inf
        by = parts.masked_fill(~keep[:, :, None], -math.inf).reshape(z.shape)
    picks = []
    for _ in range(case["k"]):
        best = by.argmax(1)
        picks.append(best)
        by[rows, best] = -math.inf
    w = torch.stack([prob[rows, b] for b in picks], dim=1)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    r = {"weights": w.detach(), "ids": None}
    if case["train"]:
        r["load"] = None
        r["grad"], = torch.autograd.grad(w, z, s["g_weights"].double())
    return r


def _exact_balance(case, s):
    z = s["logits"].double()
    u = (torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, dim=1)) / case["eps"]
    n, e = u.shape
    g = torch.zeros(e, dtype=torch.float64, device=u.device)
    for _ in range(case["n_iters"]):
        f = math.log(e) - torch.logsumexp(u + g, dim=1)
        g = math.log(n) - torch.logsumexp(u + f[:, None], dim=0)
    return {"f": case["eps"] * f, "g": case["eps"] * g}
