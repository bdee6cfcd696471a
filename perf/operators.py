"""Cases of the training operators (attention with capped, biased and masked scores; layer norm;
AdamW over many tensors): their inputs, their plain forms and what one pass cannot do without.

A case is a dict of plain values.  `run` computes a case in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or, where `own` is true, through this
package's entry points.  `exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 256                     # elements of an 8-bit state that share a scale


# ---------------------------------------------------------------- cases

def attention_case(name, B, Hq, Hkv, Sq, Skv, D, dtype="bf16", train=False, causal=True, softcap=0.0, alibi=False,
                   docs=0, pad=0, prefix=False, token_major=False):
    return {"name": name, "op": "attention", "B": B, "Hq": Hq, "Hkv": Hkv, "Sq": Sq, "Skv": Skv, "D": D, "dtype": dtype,
            "train": train, "causal": causal, "softcap": softcap, "alibi": alibi, "docs": docs, "pad": pad,
            "prefix": prefix, "token_major": token_major}


def norm_case(name, rows, cols, dtype, weight, train=True, gap=0):
    return {"name": name, "op": "layer_norm", "rows": rows, "cols": cols, "dtype": dtype, "weight": weight,
            "train": train, "gap": gap}


def adamw_case(name, sizes, dtype="f32", bits=32):
    return {"name": name, "op": "adamw", "sizes": " ".join(str(n) for n in sizes), "dtype": dtype, "bits": bits}


def block_sizes(width, layers, vocab):
    """Parameter sizes of a decoder: an embedding, then per layer two norms, the attention's
    projections and a feed-forward pair four times as wide."""
    one = [width, width, 3 * width * width, width * width, width, width, 4 * width * width, 4 * width * width]
    return [vocab * width] + one * layers


def listed():
    return [
        # one token of eight requests against their caches, distance bias: serving
        attention_case("attention_token", 8, 32, 8, 1, 8192, 128, causal=True, alibi=True),
        # the smallest training call: a test-sized model, latency
        attention_case("attention_small_train", 1, 4, 2, 96, 96, 64, train=True, softcap=30.0),
        # the long-context causal workload of the benchmark, with capped scores: prompt processing
        attention_case("attention_long", 1, 16, 16, 4096, 4096, 128, softcap=30.0),
        # the same workload as a training step
        attention_case("attention_long_train", 1, 16, 16, 4096, 4096, 128, train=True, softcap=30.0),
        # documents packed into one row, shared key/value heads, padding at the end, projections' token-major layout
        attention_case("attention_packed_train", 1, 16, 4, 6145, 6145, 128, train=True, docs=7, pad=45,
                       token_major=True),
        # prefix language modelling in f16 at an odd length and a narrow head, distance bias
        attention_case("attention_prefix_train", 3, 6, 6, 777, 777, 80, "f16", train=True, alibi=True, prefix=True),
        # a few rows: one decoding step's norm
        norm_case("norm_few_rows", 16, 1024, "bf16", "bf16", train=False),
        # a training step's norm, f32 weights under bf16 activations
        norm_case("norm_train", 8192, 4096, "bf16", "f32"),
        # odd width and row count, rows of a wider buffer
        norm_case("norm_odd_train", 3001, 5003, "f32", "f32", gap=5),
        # a test-sized model: latency
        adamw_case("adamw_small", block_sizes(64, 2, 500)),
        # a decoder's parameters with f32 states
        adamw_case("adamw_large", block_sizes(2048, 4, 32000)),
        # bf16 parameters with 8-bit states, sizes that end inside a block
        adamw_case("adamw_8bit", [n + 7 * (i % 3) for i, n in enumerate(block_sizes(1536, 4, 20011))], "bf16", 8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "layer_norm", "adamw"])
    if kind == "attention":
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 1, 2, 4, 5])
        B = rng.choice([1, 1, 2, 3, 8])
        D = rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 128])
        token = rng.random() < 0.25
        train = not token and rng.random() < 0.6
        Skv = _log(rng, 16 if train else 1, 8192)
        while B * Hq * Skv * Skv > 1 << 28 and not token:
            Skv = Skv * 2 // 3
        Sq = (min(Skv, rng.choice([1, 1, 2, 5])) if token else Skv if rng.random() < 0.8
              else max(Skv // 2 + 1, Skv - rng.randrange(1, 40)))
        causal = token or rng.random() < 0.75
        docs = 0 if rng.random() < 0.6 else min(rng.choice([1, 2, 5, 12]), max(1, Skv // 8))
        pad = 0 if docs == 0 or token else rng.choice([0, 3, Skv // 8])
        prefix = causal and not token and rng.random() < 0.3
        c = attention_case("", B, Hq, Hkv, Sq, Skv, D, rng.choice(["bf16", "bf16", "f16"]), train, causal,
                           rng.choice([0.0, 0.0, 20.0, 30.0, 50.0]), rng.random() < 0.4, docs, pad, prefix,
                           rng.random() < 0.4)
    elif kind == "layer_norm":
        cols = _log(rng, 8, 16384)
        rows = max(1, _log(rng, 1, min(16384, (1 << 25) // cols)))
        dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
        c = norm_case("", rows, cols, dtype, rng.choice([dtype, "f32"]), rng.random() < 0.75, rng.choice([0, 0, 3, 8]))
    else:
        n = rng.choice([1, 3, 8, 20, 40])
        sizes = [_log(rng, 1, 1 << 22) for _ in range(n)]
        c = adamw_case("", sizes, rng.choice(["f32", "bf16", "f16"]), rng.choice([8, 32]))
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def doc_ids(case):
    """[B, Skv] document of each token, -1 for padding: consecutive documents whose lengths differ."""
    S, n, pad = case["Skv"], case["docs"], case["pad"]
    used = max(0, S - pad)
    cuts = np.cumsum(1.0 + 0.5 * (np.arange(n) % 3))
    cuts = np.floor(used * cuts / cuts[-1]).astype(np.int64)
    ids = np.searchsorted(cuts, np.arange(S), side="right").astype(np.int32)
    ids[used:] = -1
    return np.broadcast_to(ids, (case["B"], S)).copy()


def prefix_lengths(case):
    return (case["Skv"] // 4 + 7 * np.arange(case["B"])).clip(0, case["Skv"]).astype(np.int32)


def slopes_of(case):
    """Geometric slopes, one for each query head."""
    return 2.0 ** (-8.0 * np.arange(1, case["Hq"] + 1) / case["Hq"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "attention":
        B, Hq, Hkv, Sq, Skv, D = (case[k] for k in ("B", "Hq", "Hkv", "Sq", "Skv", "D"))

        def normal(H, S, heavy=False):
            shape = (B, S, H, D) if case["token_major"] else (B, H, S, D)
            x = torch.randn(shape, device="cuda", generator=g)
            x = x.transpose(1, 2) if case["token_major"] else x
            if heavy:       # a hundredth of the keys eight times as long, as in the long-context workload
                x = torch.where(torch.rand(B, H, S, 1, device="cuda", generator=g) < 0.01, x * 8, x)
                x = x.transpose(1, 2).contiguous().transpose(1, 2) if case["token_major"] else x.contiguous()
            return x.to(dt)
        s["q"], s["k"], s["v"] = normal(Hq, Sq), normal(Hkv, Skv, True), normal(Hkv, Skv)
        if case["train"]:
            s["grad"] = normal(Hq, Sq)
        s["kw"] = {"causal": case["causal"], "softcap": case["softcap"]}
        if case["alibi"]:
            s["kw"]["slopes"] = torch.tensor(slopes_of(case), dtype=torch.float32, device="cuda")
        if case["docs"]:
            s["kw"]["docs"] = torch.tensor(doc_ids(case), device="cuda")
        if case["prefix"]:
            s["kw"]["prefix"] = torch.tensor(prefix_lengths(case), device="cuda")
    elif case["op"] == "layer_norm":
        n, w, gap = case["rows"], case["cols"], case["gap"]
        wt = TYPES[case["weight"]]

        def rows():
            return (torch.randn(n, w + gap, device="cuda", generator=g) * 2 + 0.5).to(dt)[:, :w]
        s["x"] = rows()
        s["weight"] = (1 + 0.2 * torch.randn(w, device="cuda", generator=g)).to(wt)
        s["bias"] = (0.2 * torch.randn(w, device="cuda", generator=g)).to(wt)
        if case["train"]:
            s["grad"] = torch.randn(n, w, device="cuda", generator=g).to(dt)
    else:
        sizes = [int(n) for n in case["sizes"].split()]
        s["params"] = [(0.02 * torch.randn(n, device="cuda", generator=g)).to(dt) for n in sizes]
        s["grads"] = [(1e-3 * torch.randn(n, device="cuda", generator=g)).to(dt) for n in sizes]
        # the states lie in one buffer, each tensor's from a multiple of BLOCK on
        room = sum(-(-n // BLOCK) * BLOCK for n in sizes)
        m = 3e-4 * torch.randn(room, device="cuda", generator=g)
        v = torch.rand(room, device="cuda", generator=g) * 1e-6 + 1e-9
        if case["bits"] == 8:
            s["m"], s["m_scale"] = to_8bit(m, False)
            s["v"], s["v_scale"] = to_8bit(v.sqrt(), True)
        else:
            s["m"], s["v"] = m, v
        s["step"] = 100
    return s


HYPER = {"lr": 1e-3, "betas": (0.9, 0.95), "eps": 1e-8, "weight_decay": 0.1}


# ---------------------------------------------------------------- plain forms

def visible(case, kw, device):
    """[B or 1, Sq, Skv] truth values: whether query i sees key j."""
    Sq, Skv = case["Sq"], case["Skv"]
    j = torch.arange(Skv, device=device)
    i = torch.arange(Sq, device=device)[:, None] + (Skv - Sq)
    see = torch.ones(1, Sq, Skv, dtype=torch.bool, device=device)
    if case["causal"]:
        see = (j <= i)[None]
        if "prefix" in kw:
            see = see | (j < kw["prefix"][:, None, None])
    if "docs" in kw:
        d = kw["docs"]
        mine = d[:, Skv - Sq:, None]
        see = see & (mine == d[:, None, :]) & (mine >= 0)
    return see


def plain_attention(s):
    case, kw = s["case"], s["kw"]
    B, Hq, Hkv, Sq, Skv, D = (case[k] for k in ("B", "Hq", "Hkv", "Sq", "Skv", "D"))
    dt, cap = TYPES[case["dtype"]], case["softcap"]
    scale = 1.0 / math.sqrt(D)
    q = s["q"].float().reshape(B, Hkv, Hq // Hkv, Sq, D)
    k = s["k"].float()[:, :, None]
    v = s["v"].float()[:, :, None]
    see = visible(case, kw, q.device)[:, None, None]
    t = q @ k.transpose(-1, -2) * scale
    th = None
    if cap:
        th = torch.tanh(t / cap)
        t = th * cap
    if "slopes" in kw:
        away = (torch.arange(Sq, device=q.device)[:, None] + (Skv - Sq) - torch.arange(Skv, device=q.device)).abs()
        t = t - kw["slopes"].reshape(1, Hkv, Hq // Hkv, 1, 1) * away
    t = torch.where(see, t, -math.inf)
    top = t.amax(-1, keepdim=True)
    p = torch.exp(t - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = p @ v
    answer = {"out": out.reshape(B, Hq, Sq, D).to(dt)}
    if case["train"]:
        go = s["grad"].float().reshape(B, Hkv, Hq // Hkv, Sq, D)
        dv = (p.transpose(-1, -2) @ go).sum(2)
        dp = go @ v.transpose(-1, -2)
        ds = p * (dp - (dp * p).sum(-1, keepdim=True))
        if cap:
            ds = ds * (1 - th * th)
        answer["dq"] = (ds @ k * scale).reshape(B, Hq, Sq, D).to(dt)
        answer["dk"] = (ds.transpose(-1, -2) @ q * scale).sum(2).to(dt)
        answer["dv"] = dv.to(dt)
    return answer


def plain_norm(s):
    x, w = s["x"].float(), s["weight"].float()
    dt, wt = s["x"].dtype, s["weight"].dtype
    d = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-5)
    h = d * r
    answer = {"y": (h * w + s["bias"].float()).to(dt)}
    if "grad" in s:
        dy = s["grad"].float()
        a = dy * w
        answer["dx"] = (r * (a - a.mean(-1, keepdim=True) - h * (a * h).mean(-1, keepdim=True))).to(dt)
        answer["dw"] = (dy * h).sum(0).to(wt)
        answer["db"] = dy.sum(0).to(wt)
    return answer


def to_8bit(x, positive):
    """e4m3 values and a scale for each BLOCK of x; with `positive`, a value above zero never becomes zero."""
    b = x.reshape(-1, BLOCK)
    top = b.abs().amax(1)
    live = top >= 2.0 ** -100
    scale = torch.where(live, top / 448.0, 0.0)
    back = torch.where(live, 448.0 / top, 0.0)
    c = b * back[:, None]
    if positive:
        c = torch.where((c > 0) & (c < 2.0 ** -9), 2.0 ** -9, c)
    return c.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).reshape(-1), scale


def from_8bit(c, scale):
    return (c.float().reshape(-1, BLOCK) * scale[:, None]).reshape(-1)


def plain_adamw(s):
    """Every operation rounded to 32 bits by itself, the states read and written in their form."""
    b1, b2 = HYPER["betas"]
    s["step"] += 1
    t, eight = s["step"], s["case"]["bits"] == 8
    f = lambda x: float(np.float32(x))  # noqa: E731
    keep = f(1 - HYPER["lr"] * HYPER["weight_decay"])
    rate = f(HYPER["lr"] / (1 - b1 ** t))
    undo = f(1 / math.sqrt(1 - b2 ** t))

    def flat(ts):       # in one row, each tensor from a multiple of BLOCK on
        return torch.cat([torch.nn.functional.pad(x.float(), (0, -x.numel() % BLOCK)) for x in ts])
    g, p = flat(s["grads"]), flat(s["params"])
    m, v = s["m"], s["v"]
    if eight:
        m, r = from_8bit(m, s["m_scale"]), from_8bit(v, s["v_scale"])
        v = r * r
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    root = torch.sqrt(v)
    p = p * keep - (m / (root * undo + f(HYPER["eps"]))) * rate
    starts = np.concatenate([[0], np.cumsum([-(-x.numel() // BLOCK) * BLOCK for x in s["params"]])])
    torch._foreach_copy_(s["params"], [p[a:a + x.numel()] for a, x in zip(starts.tolist(), s["params"])])
    # what lies between the tensors is no element: it stays as it is, for 8-bit blocks zero
    live = torch.cat([torch.nn.functional.pad(torch.ones_like(x, dtype=torch.bool), (0, -x.numel() % BLOCK)) for x in s["params"]])
    if eight:
        m, root = torch.where(live, m, 0.0), torch.where(live, root, 0.0)
        m, m_scale = to_8bit(m, False)
        v, v_scale = to_8bit(root, True)
        s["m_scale"].copy_(m_scale)
        s["v_scale"].copy_(v_scale)
    else:
        m, v = torch.where(live, m, s["m"]), torch.where(live, v, s["v"])
    s["m"].copy_(m)
    s["v"].copy_(v)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        import bitwise_deterministic_shard_gb300 as da
        if op == "attention":
            q, k, v = state["q"], state["k"], state["v"]
            if "grad" not in state:
                return {"out": da.attention(q, k, v, **state["kw"])}
            out, lse = da.attention_forward(q, k, v, **state["kw"])
            dq, dk, dv = da.attention_backward(q, k, v, out, lse, state["grad"], **state["kw"])
            return {"out": out, "dq": dq, "dk": dk, "dv": dv}
        if op == "layer_norm":
            x, w, b = state["x"], state["weight"], state["bias"]
            if "grad" not in state:
                return {"y": da.layer_norm(x, w, b)}
            y, mean, rstd = da.layer_norm_forward(x, w, b)
            dx, dw, db = da.layer_norm_backward(state["grad"], x, w, mean, rstd)
            return {"y": y, "dx": dx, "dw": dw, "db": db}
        state["step"] += 1
        da.adamw_step(state["params"], state["grads"], state["m"], state["v"], state["step"],
                      exp_avg_scale=state.get("m_scale"), exp_avg_sq_scale=state.get("v_scale"), **HYPER)
    elif op == "attention":
        return plain_attention(state)
    elif op == "layer_norm":
        return plain_norm(state)
    else:
        plain_adamw(state)
    return {k: state[k] for k in ("params", "m", "v", "m_scale", "v_scale") if k in state}


# ---------------------------------------------------------------- what a pass cannot do without

def pairs_of(case):
    """Pairs of a query and a key that it sees, of one head, over the batch."""
    Sq, Skv = case["Sq"], case["Skv"]
    pos = np.arange(Skv - Sq, Skv)
    total = 0
    for b in range(case["B"]):
        hi = np.full(Sq, Skv)
        lo = np.zeros(Sq, dtype=np.int64)
        if case["causal"]:
            hi = pos + 1
            if case["prefix"]:
                hi = np.maximum(hi, prefix_lengths(case)[b])
        if case["docs"]:
            ids = doc_ids(case)[b]
            first = np.searchsorted(np.where(ids < 0, 1 << 30, ids), ids[pos], side="left")
            last = np.searchsorted(np.where(ids < 0, 1 << 30, ids), ids[pos], side="right")
            lo, hi = np.where(ids[pos] < 0, 0, first), np.where(ids[pos] < 0, 0, np.minimum(hi, last))
        total += int(np.maximum(hi - lo, 0).sum())
    return total


def work(case):
    if case["op"] == "attention":
        B, Hq, Hkv, Sq, Skv, D = (case[k] for k in ("B", "Hq", "Hkv", "Sq", "Skv", "D"))
        q, kv = 2 * B * Hq * Sq * D, 2 * B * Hkv * Skv * D
        products = 7 if case["train"] else 2      # forward 2, backward 5
        return {"bytes": (4 * q + 4 * kv) if case["train"] else 2 * q + 2 * kv,
                "flops": 2 * products * D * Hq * pairs_of(case)}
    if case["op"] == "layer_norm":
        n, w = case["rows"], case["cols"]
        es, ws = (4 if case[k] == "f32" else 2 for k in ("dtype", "weight"))
        return {"bytes": n * w * es * (4 if case["train"] else 2) + w * ws * (4 if case["train"] else 2),
                "flops": n * w * (22 if case["train"] else 8)}
    n = sum(int(x) for x in case["sizes"].split())
    es = 4 if case["dtype"] == "f32" else 2
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (3 * es + state), "flops": 15 * n}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return exact_attention(case, s)
    if case["op"] == "layer_norm":
        x, w, b = (s[k].double().requires_grad_(case["train"]) for k in ("x", "weight", "bias"))
        var, mean = torch.var_mean(x, -1, correction=0, keepdim=True)
        y = (x - mean) * (var + 1e-5) ** -0.5 * w + b
        if not case["train"]:
            return {"y": y}
        dx, dw, db = torch.autograd.grad(y, (x, w, b), s["grad"].double())
        return {"y": y.detach(), "dx": dx, "dw": dw, "db": db}
    return exact_adamw(case, s)


def exact_attention(case, s):
    B, Hq, Hkv, Sq, Skv = (case[k] for k in ("B", "Hq", "Hkv", "Sq", "Skv"))
    kw, dev = s["kw"], s["q"].device
    G = Hq // Hkv
    names = ("out", "dq", "dk", "dv") if case["train"] else ("out",)
    r = {n: torch.zeros(s[k].shape, dtype=torch.float64, device=dev) for n, k in zip(names, ("q", "q", "k", "v"))}
    row = np.arange(Skv - Sq, Skv)
    col = np.arange(Skv)
    for b in range(B):
        hidden = torch.zeros(Sq, Skv, dtype=torch.bool, device=dev)
        if case["causal"]:
            last = row + 1 if not case["prefix"] else np.maximum(row + 1, prefix_lengths(case)[b])
            hidden |= torch.tensor(col, device=dev)[None] >= torch.tensor(last, device=dev)[:, None]
        if case["docs"]:
            ids = torch.tensor(doc_ids(case)[b], device=dev)
            hidden |= (ids[row[0]:, None] != ids[None]) | (ids[row[0]:, None] < 0)
        gone = hidden.all(1)
        for h in range(Hq):
            q, k, v = (x.double().requires_grad_(case["train"])
                       for x in (s["q"][b, h], s["k"][b, h // G], s["v"][b, h // G]))
            score = torch.einsum("id,jd->ij", q, k) / math.sqrt(case["D"])
            if case["softcap"]:
                score = case["softcap"] * torch.tanh(score / case["softcap"])
            if case["alibi"]:
                slope = float(np.float32(slopes_of(case)[h]))
                score = score - slope * torch.tensor(np.abs(row[:, None] - col[None]), device=dev)
            score = score.masked_fill(hidden & ~gone[:, None], -math.inf)
            p = torch.softmax(score, -1).masked_fill(gone[:, None], 0.0)
            out = torch.einsum("ij,jd->id", p, v)
            r["out"][b, h] = out.detach()
            if case["train"]:
                dq, dk, dv = torch.autograd.grad(out, (q, k, v), s["grad"][b, h].double())
                r["dq"][b, h] = dq
                r["dk"][b, h // G] += dk
                r["dv"][b, h // G] += dv
    return r


def exact_adamw(case, s):
    b1, b2 = HYPER["betas"]
    t = s["step"] + 1
    eight = case["bits"] == 8
    if eight:
        m0 = s["m"].double() * s["m_scale"].double().repeat_interleave(BLOCK)
        v0 = (s["v"].double() * s["v_scale"].double().repeat_interleave(BLOCK)) ** 2
    else:
        m0, v0 = s["m"].double(), s["v"].double()
    m1, v1 = (torch.zeros_like(m0), torch.zeros_like(v0)) if eight else (m0.clone(), v0.clone())
    params, at = [], 0
    for p, g in zip(s["params"], s["grads"]):
        n = p.numel()
        p, g = p.double(), g.double()
        m = b1 * m0[at:at + n] + (1 - b1) * g
        v = b2 * v0[at:at + n] + (1 - b2) * g ** 2
        hat_m, hat_v = m / (1 - b1 ** t), v / (1 - b2 ** t)
        params.append(p - HYPER["lr"] * (HYPER["weight_decay"] * p + hat_m / (hat_v.sqrt() + HYPER["eps"])))
        m1[at:at + n], v1[at:at + n] = m, v
        at += -(-n // BLOCK) * BLOCK
    if not eight:
        return {"params": params, "m": m1, "v": v1}

    def rounded(x, positive):
        x = x.reshape(-1, BLOCK)
        top = x.abs().amax(1)
        scale = torch.where(top >= 2.0 ** -100, top / 448, 0.0)
        c = torch.where(scale[:, None] > 0, x / scale[:, None], 0.0)
        # the nearest e4m3 value: steps of 2^-3 of the binade, 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(c.abs().clamp_min(2.0 ** -6))) - 3)
        q = torch.round(c / step) * step
        if positive:
            q = torch.where((x > 0) & (q == 0) & (scale[:, None] > 0), 2.0 ** -9, q)
        return q.reshape(-1), scale
    mq, ms = rounded(m1, False)
    vq, vs = rounded(v1.sqrt(), True)
    return {"params": params, "m": mq, "v": vq, "m_scale": ms, "v_scale": vs}
