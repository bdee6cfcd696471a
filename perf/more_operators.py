"""Cases of the operators at the ends and in the middle of a decoder (embedding lookup and its gradient;
the gated feed-forward projections; log probabilities of given tokens with entropy and top
alternatives): their inputs, their plain forms and what one pass cannot do without.

A case is a dict of plain values.  `run` computes a case in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or, where `own` is true, through this
package's entry points.  `exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases

def embedding_case(name, tokens, vocab, width, dtype="bf16", train=True, scale=1.0, padding=False, ids="i64"):
    return {"name": name, "op": "embedding", "tokens": tokens, "vocab": vocab, "width": width, "dtype": dtype, "train": train,
            "scale": scale, "padding": padding, "ids": ids}


def gated_case(name, tokens, width, hidden, dtype="bf16", train=False, activation="silu"):
    return {"name": name, "op": "gated", "tokens": tokens, "width": width, "hidden": hidden, "dtype": dtype, "train": train,
            "activation": activation}


def probs_case(name, rows, vocab, dtype, top=0, train=False, temperature=1.0, masked=False, gap=0):
    return {"name": name, "op": "log_probs", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top, "train": train,
            "temperature": temperature, "masked": masked, "gap": gap}


def listed():
    return [
        # one decoding step of 64 requests: latency
        embedding_case("embedding_few", 64, 32000, 4096, train=False, scale=64.0),
        # the training batch of a large vocabulary, tokens as frequent as words are: the gradient has a row for each entry
        embedding_case("embedding_train", 16384, 128256, 2048),
        # odd width and vocabulary in f32, scaled, a tenth of the batch padding, 32-bit ids
        embedding_case("embedding_odd_train", 3001, 20011, 1003, "f32", scale=math.sqrt(1003), padding=True, ids="i32"),
        # one token of one request: the weights are read once
        gated_case("gated_token", 1, 4096, 12288),
        # one decoding step of 48 requests in f16
        gated_case("gated_batch", 48, 2048, 8192, "f16", activation="gelu_tanh"),
        # a prompt
        gated_case("gated_prompt", 4096, 4096, 12288),
        # a training step's block
        gated_case("gated_train", 8192, 2048, 8192, train=True),
        # ragged sizes with gradient, f16, the error-function activation
        gated_case("gated_odd_train", 1537, 1000, 2744, "f16", train=True, activation="gelu"),
        # one decoding step of 8 requests: the sampled tokens' log probabilities and 20 alternatives for each
        probs_case("log_probs_few", 8, 128256, "f32", top=20),
        # scoring prompts: the vocabulary-sharded workload's rows and columns, with 5 alternatives
        probs_case("log_probs_prompt", 4096, 128256, "f32", top=5),
        # a policy-gradient step with an entropy bonus on bf16 logits
        probs_case("log_probs_train", 8192, 128256, "bf16", train=True),
        # odd sizes, rows of a wider buffer, a temperature, forbidden tokens and rows without a target
        probs_case("log_probs_odd_train", 777, 32003, "f16", top=7, train=True, temperature=0.7, masked=True, gap=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["embedding", "gated", "gated", "log_probs", "log_probs"])
    if kind == "embedding":
        width = _log(rng, 8, 8192)
        vocab = _log(rng, 16, min(200000, (1 << 28) // width))
        tokens = _log(rng, 1, min(65536, (1 << 25) // width))
        c = embedding_case("", tokens, vocab, width, rng.choice(["f32", "bf16", "bf16", "f16"]), rng.random() < 0.8,
                           rng.choice([1.0, 1.0, 0.5, math.sqrt(width)]), rng.random() < 0.4, rng.choice(["i64", "i32"]))
    elif kind == "gated":
        train = rng.random() < 0.5
        width, hidden = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 1536)
        tokens = rng.choice([1, 2, 3, 5, 8, 13, 32, 100]) if not train and rng.random() < 0.5 else _log(rng, 1, 8192)
        while tokens * width * hidden > 1 << 35:
            tokens = tokens * 2 // 3
        c = gated_case("", tokens, width, hidden, rng.choice(["bf16", "bf16", "f16"]), train,
                       rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]))
    else:
        vocab = _log(rng, 8, 262144)
        rows = _log(rng, 1, min(16384, (1 << 28) // vocab))
        train = rng.random() < 0.5
        c = probs_case("", rows, vocab, rng.choice(["f32", "bf16", "bf16", "f16"]), min(vocab, rng.choice([0, 0, 1, 5, 20, 32])),
                       train, rng.choice([1.0, 1.0, 0.7, 1.3]), rng.random() < 0.3, rng.choice([0, 0, 3, 8]))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]
    s = {"case": case}

    def normal(*shape, by=1.0, to=dt):
        return (torch.randn(*shape, device="cuda", generator=g) * by).to(to)
    if case["op"] == "embedding":
        n, v, w = case["tokens"], case["vocab"], case["width"]
        # the r-th most frequent entry with a probability of about 1 / r, entries in a random order
        rank = torch.exp(torch.rand(n, device="cuda", generator=g, dtype=torch.float64) * math.log(v + 1)).long() - 1
        ids = torch.randperm(v, device="cuda", generator=g)[rank.clamp(0, v - 1)]
        if case["padding"]:
            ids = torch.where(torch.rand(n, device="cuda", generator=g) < 0.1, 0, ids)
        s["ids"] = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
        s["weight"] = normal(v, w, by=0.02)
        s["padding"] = 0 if case["padding"] else None
        if case["train"]:
            s["grad"] = normal(n, w)
    elif case["op"] == "gated":
        n, w, h = case["tokens"], case["width"], case["hidden"]
        s["x"] = normal(n, w)
        s["w_gate"], s["w_up"] = normal(h, w, by=w ** -0.5), normal(h, w, by=w ** -0.5)
        if case["train"]:
            s["grad"] = normal(n, h)
    else:
        n, v = case["rows"], case["vocab"]
        x = normal(n, v + case["gap"], by=2.5, to=torch.float32)
        if case["masked"]:      # a fifth of the tokens is forbidden; in one row (where there are more) every one
            x = torch.where(torch.rand(x.shape, device="cuda", generator=g) < 0.2, -math.inf, x)
            if n > 1:
                x[n // 2] = -math.inf
        s["logits"] = x.to(dt)[:, :v]
        # sampled tokens: mostly likely ones; a row without a target has -1
        best = s["logits"].argmax(1)
        other = torch.randint(0, v, (n,), device="cuda", generator=g)
        t = torch.where(torch.rand(n, device="cuda", generator=g) < 0.6, best, other)
        if case["masked"]:
            t = torch.where(torch.rand(n, device="cuda", generator=g) < 0.1, -1, t)
        s["targets"] = t
        if case["train"]:
            s["grad"], s["grad_entropy"] = normal(n, to=torch.float32), 0.01 * normal(n, to=torch.float32)
    return s


# ---------------------------------------------------------------- plain forms

def plain_embedding(s):
    case, w, ids = s["case"], s["weight"], s["ids"].long()
    answer = {"y": (w[ids].float() * case["scale"]).to(w.dtype)}
    if case["train"]:
        go = s["grad"].float()
        if s["padding"] is not None:
            go = torch.where((ids == s["padding"])[:, None], 0.0, go)
        dw = torch.zeros(w.shape, device=w.device).index_add_(0, ids, go)
        answer["dweight"] = (dw * case["scale"]).to(w.dtype)
    return answer


def activated(g, kind):
    """act(g) and its derivative, in g's type."""
    if kind == "silu":
        z = 1 / (1 + torch.exp(-g))
        return g * z, z * (1 + g * (1 - z))
    if kind == "gelu":
        z = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * z, z + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    return torch.where(g > 0, g, 0.0), (g > 0).to(g.dtype)


def plain_gated(s):
    case, dt = s["case"], s["x"].dtype
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    g, u = x @ wg.T, x @ wu.T
    a, da = activated(g, case["activation"])
    answer = {"h": (a * u).to(dt)}
    if case["train"]:
        go = s["grad"].float()
        dg, du = go * u * da, go * a
        answer["dx"] = (dg @ wg + du @ wu).to(dt)
        answer["dw_gate"], answer["dw_up"] = (dg.T @ x).to(dt), (du.T @ x).to(dt)
    return answer


def plain_log_probs(s):
    case, t = s["case"], s["targets"]
    n, k = case["rows"], case["top"]
    z = s["logits"].float() / case["temperature"]
    m = z.amax(1, keepdim=True)
    dead = m == -math.inf
    d = z - torch.where(dead, 0.0, m)
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(torch.where(dead, 1.0, total))
    p = e / torch.where(dead, 1.0, total)
    lp = d - log_total                                     # -inf where the logit is
    lp_or_0 = torch.where(p > 0, lp, 0.0)
    entropy = -(p * lp_or_0).sum(1)
    asked = t >= 0
    answer = {"log_probs": torch.where(asked, lp.gather(1, t.clamp_min(0)[:, None])[:, 0], 0.0), "entropy": entropy}
    if k:
        # the largest first, equal ones by their index: whole numbers that order like (logit, -index)
        bits = (s["logits"].float() + 0.0).view(torch.int32).long()
        order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        index = torch.arange(case["vocab"], device=z.device)
        keys = torch.topk(order * (1 << 20) + ((1 << 20) - 1 - index), k, dim=1).values
        answer["top_indices"] = (1 << 20) - 1 - (keys & ((1 << 20) - 1))
        answer["top_log_probs"] = lp.gather(1, answer["top_indices"])
    if case["train"]:
        a, b = torch.where(asked, s["grad"], 0.0)[:, None], s["grad_entropy"][:, None]
        dx = -p * (a + b * (lp_or_0 + entropy[:, None]))
        dx = dx.scatter_add(1, t.clamp_min(0)[:, None], torch.where(dead, 0.0, a))
        answer["dlogits"] = (dx / case["temperature"]).to(s["logits"].dtype)
    return answer


# ---------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import bitwise_deterministic_shard_gb300 as da
        if op == "embedding":
            ids, w = state["ids"], state["weight"]
            answer = {"y": da.embedding_forward(ids, w, case["scale"])}
            if "grad" in state:
                answer["dweight"] = da.embedding_backward(state["grad"], ids, case["vocab"], case["scale"], state["padding"])
            return answer
        if op == "gated":
            x, wg, wu, act = state["x"], state["w_gate"], state["w_up"], case["activation"]
            if "grad" not in state:
                return {"h": da.gated_linear(x, wg, wu, act)}
            h, saved = da.gated_linear_forward(x, wg, wu, act)
            dx, dwg, dwu = da.gated_linear_backward(state["grad"], x, wg, wu, saved)
            return {"h": h, "dx": dx, "dw_gate": dwg, "dw_up": dwu}
        x, t, temperature = state["logits"], state["targets"], case["temperature"]
        r, saved = da.log_probs_forward(x, t, temperature, case["top"])
        answer = {"log_probs": r.log_probs, "entropy": r.entropy}
        if case["top"]:
            answer["top_indices"], answer["top_log_probs"] = r.top_indices, r.top_log_probs
        if "grad" in state:
            answer["dlogits"] = da.log_probs_backward(x, t, saved, state["grad"], state["grad_entropy"], temperature)
        return answer
    return {"embedding": plain_embedding, "gated": plain_gated, "log_probs": plain_log_probs}[op](state)


# ---------------------------------------------------------------- what a pass cannot do without

def distinct(n, v):
    """Entries of v that n tokens drawn as in prepare name, on average."""
    r = np.arange(1, v + 1, dtype=np.float64)
    p = np.log((r + 1) / r) / math.log(v + 1)
    return float((1 - (1 - p) ** n).sum())


def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "embedding":
        n, v, w = case["tokens"], case["vocab"], case["width"]
        ids = n * (4 if case["ids"] == "i32" else 8)
        forward = ids + (distinct(n, v) + n) * w * es
        return {"bytes": forward + ((n + v) * w * es if case["train"] else 0), "flops": n * w * (2 if case["train"] else 1)}
    if case["op"] == "gated":
        n, w, h = case["tokens"], case["width"], case["hidden"]
        x, weights, hidden = n * w * es, 2 * w * h * es, n * h * es
        return {"bytes": x + weights + hidden + (x + weights + hidden if case["train"] else 0),
                "flops": (12 if case["train"] else 4) * n * w * h}
    n, v = case["rows"], case["vocab"]
    return {"bytes": n * v * es * (2 if case["train"] else 1) + n * (16 + 12 * case["top"] + (8 if case["train"] else 0)),
            "flops": n * v * (12 if case["train"] else 6)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embedding":
        w, ids = s["weight"].double(), s["ids"].reshape(-1).long()
        r = {"y": torch.index_select(w, 0, ids) * case["scale"]}
        if case["train"]:
            dw = torch.zeros_like(w)
            order = torch.argsort(ids, stable=True)
            if case["padding"]:
                order = order[ids[order] != 0]
            if order.numel():
                names, counts = torch.unique_consecutive(ids[order], return_counts=True)
                at = torch.arange(names.numel(), device=ids.device).repeat_interleave(counts)
                sums = torch.zeros(names.numel(), w.shape[1], dtype=torch.float64, device=w.device)
                dw[names] = sums.index_add(0, at, s["grad"][order].double()) * case["scale"]
            r["dweight"] = dw
        return r
    if case["op"] == "gated":
        x, wg, wu = (s[k].double().requires_grad_(case["train"]) for k in ("x", "w_gate", "w_up"))
        g = torch.einsum("td,fd->tf", x, wg)
        kind = case["activation"]
        if kind == "silu":
            a = torch.nn.functional.silu(g)
        elif kind == "relu":
            a = torch.relu(g)
        else:
            a = torch.nn.functional.gelu(g, approximate="tanh" if kind == "gelu_tanh" else "none")
        h = a * torch.einsum("td,fd->tf", x, wu)
        if not case["train"]:
            return {"h": h}
        dx, dwg, dwu = torch.autograd.grad(h, (x, wg, wu), s["grad"].double())
        return {"h": h.detach(), "dx": dx, "dw_gate": dwg, "dw_up": dwu}
    z = s["logits"].double() / case["temperature"]
    t = s["targets"]
    lp = torch.log_softmax(z, 1)
    gone = torch.isneginf(z).all(1)
    lp = lp.masked_fill(torch.isneginf(z) | gone[:, None], -math.inf)
    p = lp.exp()
    entropy = torch.special.entr(p).sum(1)
    took = torch.take_along_dim(lp, t.clamp(min=0)[:, None], 1)[:, 0]
    r = {"log_probs": took.masked_fill(t < 0, 0.0), "entropy": entropy}
    if case["top"]:
        r["top_indices"] = None
        r["top_log_probs"] = torch.sort(lp, dim=1, descending=True).values[:, :case["top"]]
    if case["train"]:
        a, b = s["grad"].double().masked_fill(t < 0, 0.0), s["grad_entropy"].double()
        finite = lp.masked_fill(torch.isneginf(lp), 0.0)
        grad = -a[:, None] * p - b[:, None] * (p * finite + p * entropy[:, None])
        rows = torch.nonzero((t >= 0) & ~gone)[:, 0]
        grad[rows, t[rows]] += a[rows]
        r["dlogits"] = grad / case["temperature"]
    return r
