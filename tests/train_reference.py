"""Plain 64-bit forms of the training operators, and how far a kernel that rounds as documented may be
from them.

The bounds count roundings: u = eps / 2 of the 16-bit type for each rounding to it, and E = 2^-16 for
what binary32 leaves (sums of up to 2^14 terms in blocks, scores of magnitude up to 2^6 whose
error is that of their exponential, ex2 and the capped score at 2^-21)."""
import math

import torch

E = 2.0 ** -16


def attention(q, k, v, go, causal=False, scale=None, softcap=0.0, slopes=None, docs=None, prefix=None):
    q, k, v, go = (t.double() for t in (q, k, v, go))
    B, Hq, Sq, D = q.shape
    Hkv, Skv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    kk, vv = (t.repeat_interleave(G, 1) for t in (k, v))
    t = scale * (q @ kk.mT)
    c = torch.ones_like(t)
    if softcap:
        th = torch.tanh(t / softcap)
        t, c = softcap * th, 1 - th * th
    pos = torch.arange(Sq, device=q.device)[:, None] + Skv - Sq
    j = torch.arange(Skv, device=q.device)[None]
    if slopes is not None:
        t = t - slopes.double()[None, :, None, None] * (pos - j).abs()
    see = torch.ones(B, 1, Sq, Skv, dtype=torch.bool, device=q.device)
    if causal:
        see = see & (j <= pos)
        if prefix is not None:
            see = see | (j < prefix.long()[:, None, None, None])
    if docs is not None:
        mine = docs[:, Skv - Sq:]
        see = see & ((mine[:, :, None] == docs[:, None, :]) & (mine[:, :, None] >= 0))[:, None]
    see = see.expand(B, Hq, Sq, Skv)
    t = torch.where(see, t, -math.inf)
    lse = torch.logsumexp(t, -1) if Skv else torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device=q.device)
    p = torch.where(see, torch.exp(t - torch.where(lse == -math.inf, 0.0, lse)[..., None]), 0.0)
    out = p @ vv
    dp = go @ vv.mT
    delta = (p * dp).sum(-1, keepdim=True)
    ds = p * c * (dp - delta)

    def heads(x):
        return x.reshape(B, Hkv, G, *x.shape[2:]).sum(2)
    a = ds.abs()
    off = (out.abs() * go.abs()).sum(-1, keepdim=True)     # times u: how far delta from the rounded output is off
    rough = p * (dp.abs() + delta.abs())
    return {"out": out, "lse": lse, "dq": scale * (ds @ kk), "dk": scale * heads(ds.mT @ q), "dv": heads(p.mT @ go),
            "abs": {"out": p @ vv.abs(), "dv": heads(p.mT @ go.abs()), "dk": abs(scale) * heads(a.mT @ q.abs()),
                    "dq": abs(scale) * (a @ kk.abs()), "dq_off": abs(scale) * off * ((p * c) @ kk.abs()),
                    "dk_rough": abs(scale) * heads(rough.mT @ q.abs()), "dq_rough": abs(scale) * (rough @ kk.abs())}}


def attention_tolerance(r, dtype):
    u = torch.finfo(dtype).eps / 2
    A = r["abs"]
    tiny = 2.0 ** -24 if dtype == torch.float16 else 0.0     # half of the smallest f16 step, per weight and result
    tol = {"out": u * (r["out"].abs() + A["out"]) + E * A["out"],
           "dv": u * (r["dv"].abs() + A["dv"]) + E * A["dv"],
           "dk": u * (r["dk"].abs() + A["dk"]) + E * A["dk_rough"],
           # ds is rounded with the rough delta, and so is E's weight: twice u for what the correction takes back
           "dq": u * (r["dq"].abs() + A["dq"]) + 2 * u * u * A["dq_off"] + E * A["dq_rough"]}
    n = {"out": 1.0, "dv": 1.0, "dk": 1.0, "dq": 1.0}
    return {k: 1.02 * t + tiny * 40 * n[k] + 1e-30 for k, t in tol.items()}


def layer_norm(x, w, b, dy, eps=1e-5):
    x, dy = x.double(), dy.double()
    w = torch.ones(x.shape[-1], dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros_like(w) if b is None else b.double()
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    h = (x - mean) * rstd
    a = dy * w
    s1, s2 = a.mean(-1, keepdim=True), (a * h).mean(-1, keepdim=True)
    return {"y": h * w + b, "dx": rstd * (a - s1 - h * s2), "dw": (dy * h).sum(0), "db": dy.sum(0), "mean": mean, "rstd": rstd,
            "abs": {"h": (x.abs() + x.abs().mean(-1, keepdim=True)) * rstd, "w": w.abs(), "b": b.abs(),
                    "dx": rstd * (a.abs() + a.abs().mean(-1, keepdim=True) + h.abs() * (a * h).abs().mean(-1, keepdim=True)),
                    "dw": (dy * h).abs().sum(0), "db": dy.abs().sum(0), "dy": dy.abs(), "a": a.abs(), "hh": h.abs()}}


def layer_norm_tolerance(r, dtype, wdtype, rows, cols):
    """k roundings of binary32 at the longest chain of a row's sums (a thread's 32 terms, or its share of a
    wider row, and the tree), n at the longest of a column's."""
    e = 2.0 ** -24
    k, n = 48 + cols / 1024, 48 + rows / 300 + 1300 / 32
    A = r["abs"]
    u = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    uw = e if wdtype == torch.float32 else torch.finfo(wdtype).eps / 2
    h = k * e * A["h"]                                       # of the normalised value, its variance's error with it
    h = h + k * e * A["hh"]
    dx = u * r["dx"].abs() + 3 * k * e * A["dx"] + r["rstd"] * (
        h * (A["a"] * A["hh"]).mean(-1, keepdim=True) + A["hh"] * (A["a"] * h).mean(-1, keepdim=True))
    tol = {"y": u * r["y"].abs() + h * A["w"] + 4 * e * (A["hh"] * A["w"] + A["b"]), "dx": dx,
           "dw": uw * r["dw"].abs() + n * e * A["dw"] + (A["dy"] * h).sum(0), "db": uw * r["db"].abs() + n * e * A["db"]}
    floor = 2.0 ** -25 if dtype == torch.float16 else 0.0    # half of f16's smallest step
    wfloor = 2.0 ** -25 if wdtype == torch.float16 else 0.0
    return {k_: 1.02 * t + (floor if k_ in ("y", "dx") else wfloor) + 1e-30 for k_, t in tol.items()}
