"""Plain 64-bit forms of the operators at the ends and in the middle of a decoder, and how far a kernel that rounds
as documented may be from them.

u: half a step of a 16-bit type (bf16 2^-8, f16 2^-11), e = 2^-24 that of binary32.  ex2, rcp and the like are off by some 2^-22;
every bound counts the roundings on the longest way of a value and is multiplied by 1.02 for the products of two roundings."""
import math

import torch

e = 2.0 ** -24
INF = float("inf")


def half_step(dtype):
    return e if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def least(dtype):
    """Half of the type's smallest step."""
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


# ---------------------------------------------------------------- embedding

def embedding(ids, weight, dy, scale=1.0, padding_idx=None):
    w, dy, flat = weight.double(), dy.double().reshape(-1, weight.shape[1]), ids.reshape(-1).long()
    known = (flat >= 0) & (flat < w.shape[0])
    y = torch.where(known[:, None], scale * w[flat.clamp(0, w.shape[0] - 1)], 0.0).reshape(*ids.shape, w.shape[1])
    keep = known if padding_idx is None else known & (flat != padding_idx)
    dw, size = torch.zeros_like(w), torch.zeros_like(w)
    dw.index_add_(0, flat[keep], dy[keep])
    size.index_add_(0, flat[keep], dy[keep].abs())
    count = torch.bincount(flat[keep], minlength=w.shape[0])
    return {"y": y, "dw": scale * dw, "size": abs(scale) * size, "count": count}


def embedding_tolerance(r, dtype, scale):
    """The lookup: the product in binary32 and the type's rounding (none of them for a scale of 1).  The gradient: a chain of up to
    32 tokens, an eighth of the chunks, eight sums of those and the scale."""
    u = half_step(dtype)
    f = 2.0 ** -24 if scale != 1.0 else 0.0        # a scale that is not a binary32 number
    ty = 0.0 * r["y"].abs() if scale == 1.0 else (u + e + f) * r["y"].abs() + least(dtype)
    chain = 32 + torch.ceil(r["count"] / 256.0) + 8 + 2
    rounded = 0.0 if dtype == torch.float32 else u
    tw = chain[:, None] * e * r["size"] + (rounded + f) * r["dw"].abs() + (least(dtype) if rounded else 0.0)
    return {"y": 1.02 * ty, "dw": 1.02 * tw + 1e-300}


# ---------------------------------------------------------------- gated feed-forward

def act(g, kind):
    """act(g), act'(g), and a bound of |act''|."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s)), 0.5
    if kind == "gelu":
        z = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
        return g * z, z + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi), 0.8
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        y = 2 * c * (g + 0.044715 * g ** 3)
        s = torch.sigmoid(y)
        return g * s, s + g * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * g * g), 0.85
    return g.clamp_min(0), (g > 0).double(), 0.0


def gated(x, wg, wu, dh, kind):
    x, wg, wu, dh = (t.double() for t in (x, wg, wu, dh))
    D, F = wg.shape[1], wg.shape[0]
    g, u = x @ wg.T, x @ wu.T
    a, d, bend = act(g, kind)
    dg, du = dh * u * d, dh * a
    return {"h": a * u, "dx": dg @ wg + du @ wu, "dwg": dg.T @ x, "dwu": du.T @ x,
            "parts": (x, wg, wu, dh, g, u, a, d, bend, dg, du, D, F)}


def gated_tolerance(r, dtype, kind):
    """Sums of n products: the tensor cores add 16 at a time to a binary32 sum, each time off by at most 2^-22 of the sum of
    magnitudes; plain loads add n / 32 in a chain of binary32.  Activations: the exponent's argument is rounded (2^-24 of it, three
    times for the cubic), so e^x is off by that much of |x|, and 2^-21 for the rest."""
    x, wg, wu, dh, g, u, a, d, bend, dg, du, D, F = r["parts"]
    T = x.shape[0]
    r16, small = half_step(dtype), least(dtype)
    acc = lambda n: (n / 16 + 3) * 2.0 ** -22  # noqa: E731
    og = acc(D) * (x.abs() @ wg.abs().T)
    ou = acc(D) * (x.abs() @ wu.abs().T)
    arg = 2 * g.abs() * (1 + 0.045 * g * g) if kind == "gelu_tanh" else 0.5 * g * g if kind == "gelu" else g.abs()
    rel = 2.0 ** -21 + 2.0 ** -22 * arg.clamp_max(200.0)
    slope = 1.13 + 0.0 * g
    oa = slope * og + rel * a.abs() + 1e-36
    od = bend * og + rel * (1 + a.abs()) * (d.abs() + 1e-9) + rel * a.abs().clamp_max(1.0)
    if kind == "relu":
        oa, od = og, torch.where(g.abs() <= og, 1.0, 0.0)
    th = r16 * r["h"].abs() + oa * u.abs() + a.abs() * ou + oa * ou + small
    cut = 2.0 ** -15                                        # the saved factors
    op = od * u.abs() + d.abs() * ou + od * ou + cut * (u * d).abs()
    oq = oa + cut * a.abs()
    odg = (r16 + e) * dg.abs() + dh.abs() * op + small
    odu = (r16 + e) * du.abs() + dh.abs() * oq + small
    tx = r16 * r["dx"].abs() + odg @ wg.abs() + odu @ wu.abs() + acc(2 * F) * (dg.abs() @ wg.abs() + du.abs() @ wu.abs()) + small
    twg = r16 * r["dwg"].abs() + odg.T @ x.abs() + acc(T) * (dg.abs().T @ x.abs()) + small
    twu = r16 * r["dwu"].abs() + odu.T @ x.abs() + acc(T) * (du.abs().T @ x.abs()) + small
    return {k: 1.02 * t + 1e-30 for k, t in {"h": th, "dx": tx, "dwg": twg, "dwu": twu}.items()}


# ---------------------------------------------------------------- log probabilities

def log_probs(x, targets, temperature=1.0, top=0, a=None, b=None):
    z = x.double() / temperature
    V = z.shape[1]
    m = z.amax(1, keepdim=True)
    none = m[:, 0] == -INF
    d = z - torch.where(m == -INF, 0.0, m)             # first: beside the lowest logits the logarithm of the sum is lost in 64 bits too
    lp = torch.where(z == -INF, -INF, d - torch.log(torch.exp(d).sum(1, keepdim=True).clamp_min(1e-300)))
    p = torch.where(none[:, None], 0.0, torch.exp(lp))
    lp0 = torch.where(lp == -INF, 0.0, lp)
    H = -(p * lp0).sum(1)
    asked, there = targets >= 0, (targets >= 0) & (targets < V)
    r = {"lp": torch.where(asked, lp.gather(1, targets.clamp(0, V - 1)[:, None])[:, 0], 0.0), "H": H, "lp_all": lp, "p": p, "none": none,
         "far": (p * lp0 * lp0).sum(1) + (p * lp0.abs()).sum(1), "z": z}
    if top:
        r["top"], r["at"] = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top], None
        r["top_lp"] = lp.gather(1, r["top"])
    if a is not None or b is not None:
        a = torch.zeros_like(H) if a is None else torch.where(there, a.double(), 0.0)
        b = torch.zeros_like(H) if b is None else b.double()
        dx = -a[:, None] * p - b[:, None] * p * (lp0 + H[:, None])
        hit = torch.where(none, 0.0, a)
        dx.scatter_add_(1, targets.clamp(0, V - 1)[:, None], torch.where(there, hit, 0.0)[:, None])
        r["dx"] = dx / temperature
        r["dx_size"] = (p * (a.abs()[:, None] + b.abs()[:, None] * (lp0.abs() + H[:, None] + 1)) + 0.0) / temperature
        r["a"], r["b"] = a, b
    return r


def log_probs_tolerance(r, dtype, temperature):
    """A sum over V: a thread's terms one after the other in two lanes, then up to 24 joins of two roundings.  A row is read by one warp
    (up to 2048 columns: 64 lanes, 32 terms in each), two (up to 24008: 128 lanes, at most 188; from 1217 to 2432 rows also longer ones, V / 128), four (256 lanes: V / 256) or
    more; vectors that start before the row add 8.  Each term's exponent has three roundings (2^-24 of |ln p| each) and ex2 2^-22.
    So the sum is off by K of it and by 3 e of the mean |ln p|, and the entropy's sum by the same of its own."""
    rows, V = r["z"].shape
    K = (max(V / 128 if 1216 < rows <= 2432 else V / 256, 188) + 8 + 48) * e + 2.0 ** -21
    of_sum = K + 3 * e * r["far"]
    tl = of_sum[:, None] + 4 * e * (r["lp_all"].abs() + 1)
    tH = 2 * of_sum * (1 + r["H"]) + 4 * e * r["far"] + 8 * e * (1 + r["H"])
    tol = {"lp": of_sum + 4 * e * (r["lp"].abs() + 1), "H": tH, "lp_all": tl}
    if "dx" in r:
        rel = of_sum[:, None] + 2.0 ** -21 + 6 * e * torch.where(r["lp_all"] == -INF, 0.0, r["lp_all"].abs()).clamp_max(2000.0)
        u = 0.0 if dtype == torch.float32 else half_step(dtype)
        tol["dx"] = (u + 3 * e) * r["dx"].abs() + 2 * rel * r["dx_size"] + r["b"].abs()[:, None] * r["p"] * tH[:, None] / temperature
        tol["dx"] = tol["dx"] + least(dtype) + 1e-37 * (1 + r["a"].abs() + 2000 * r["b"].abs())[:, None] / temperature
    return {k: 1.02 * t for k, t in tol.items()}
