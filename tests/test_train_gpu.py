"""The training operators on the GPU against plain 64-bit forms, at the sizes, masks, strides and types where
they can go wrong."""
import os
import sys

import numpy as np
import pytest
import torch

import bitwise_deterministic_shard_gb300 as da

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import train_reference as R  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _close(got, want, tol, what):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {d.numel()} outside, worst {float((d / tol).nan_to_num(9e9).max())} of the tolerance"


def _attn_inputs(B, Hq, Hkv, Sq, Skv, D, dtype, seed=0, layout="bhsd", heavy=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def t(H, S):
        if layout == "bshd":
            return torch.randn(B, S, H, D, device="cuda", generator=g).to(dtype).transpose(1, 2)
        if layout == "wide":                     # a slice of a wider projection: strides larger than the sizes
            return torch.randn(B, S, H, D + 24, device="cuda", generator=g).to(dtype)[..., 8:8 + D].transpose(1, 2)
        if layout == "odd":                      # strides and starts that tensor maps cannot take
            return torch.randn(B, H, S, D + 3, device="cuda", generator=g).to(dtype)[..., 1:1 + D]
        if layout == "last":                     # the last dimension not contiguous
            return torch.randn(B, H, D, S, device="cuda", generator=g).to(dtype).transpose(2, 3)
        return torch.randn(B, H, S, D, device="cuda", generator=g).to(dtype)
    q, k, v, go = t(Hq, Sq), t(Hkv, Skv), t(Hkv, Skv), t(Hq, Sq)
    if heavy and Skv > 4:
        k[:, :, ::37] *= 4
    return q, k, v, go


def _attn_check(q, k, v, go, **kw):
    st = da.new_status()
    out, lse = da.attention_forward(q, k, v, status=st, **kw)
    dq, dk, dv = da.attention_backward(q, k, v, out, lse, go, status=st, **kw)
    assert da.read_status(st) == 0
    r = R.attention(q, k, v, go, **kw)
    tol = R.attention_tolerance(r, q.dtype)
    for got, n in ((out, "out"), (dq, "dq"), (dk, "dk"), (dv, "dv")):
        _close(got, r[n], tol[n], n)
    none = r["lse"] == -float("inf")
    assert torch.equal(none, lse == -float("inf"))
    assert ((lse.double() - r["lse"])[~none].abs() <= 2.0 ** -17 * (1 + r["lse"][~none].abs())).all()
    assert (out[none] == 0).all() and (dq[none] == 0).all()
    return out, lse, dq, dk, dv


SHAPES = [(1, 1, 1, 1, 1, 64), (2, 2, 1, 2, 2, 8), (1, 2, 2, 127, 127, 64), (1, 2, 1, 128, 128, 128), (1, 3, 3, 129, 129, 72),
          (2, 4, 2, 255, 255, 128), (1, 2, 1, 257, 257, 96), (1, 5, 1, 385, 385, 128), (2, 2, 2, 1, 640, 64),
          (1, 6, 2, 33, 300, 128), (1, 2, 1, 130, 517, 64), (1, 8, 1, 16, 513, 128), (1, 1, 1, 1500, 1500, 128)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_attention_plain(shape, causal, dtype):
    _attn_check(*_attn_inputs(*shape, dtype), causal=causal)


@pytest.mark.parametrize("shape", [(2, 4, 2, 255, 255, 128), (1, 6, 2, 33, 300, 64), (2, 4, 4, 1, 1030, 128), (1, 2, 1, 700, 700, 80)])
@pytest.mark.parametrize("opts", ["cap", "tight cap", "bias", "prefix", "docs", "all"])
def test_attention_options(shape, opts):
    B, Hq, Hkv, Sq, Skv, D = shape
    q, k, v, go = _attn_inputs(*shape, torch.bfloat16, seed=1)
    kw = {"causal": True}
    if opts in ("cap", "all"):
        kw["softcap"] = 20.0
    if opts == "tight cap":
        kw["softcap"] = 0.75                     # scores far beyond the cap: tanh at its ends
    if opts in ("bias", "all"):
        kw["slopes"] = torch.linspace(0.0, 0.6, Hq, device="cuda")
    if opts in ("prefix", "all"):
        kw["prefix"] = torch.tensor([Skv // 3, Skv + 5][:B], dtype=torch.int32, device="cuda")
    if opts in ("docs", "all"):
        ids = torch.arange(Skv) * 4 // Skv
        ids = torch.stack([ids, ids.flip(0)])[:B].int()          # one row falls instead of rising
        ids[0, Skv // 5:Skv // 5 + 9] = -1
        kw["docs"] = ids.cuda()
    _attn_check(q, k, v, go, **kw)
    if opts in ("cap", "bias", "docs"):
        _attn_check(q, k, v, go, **{**kw, "causal": False})


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(8, 12, 4, 257, 257, 128), (2, 40, 8, 385, 400, 64), (40, 4, 2, 40, 300, 96), (90, 2, 1, 1, 200, 128),
                                   (3, 30, 10, 513, 513, 72)])
@pytest.mark.parametrize("opts", ["plain", "cap", "all"])
def test_attention_many_heads(shape, opts, dtype):
    """Enough query tiles that each group of a CTA has one of its own (few of them share a CTA's groups)."""
    B, Hq, Hkv, Sq, Skv, D = shape
    q, k, v, go = _attn_inputs(*shape, dtype, seed=11)
    kw = {"causal": opts != "plain"}
    if opts != "plain":
        kw["softcap"] = 30.0
    if opts == "all":
        kw["slopes"] = torch.linspace(0.0, 0.4, Hq, device="cuda")
        ids = (torch.arange(Skv) * 3 // Skv).repeat(B, 1).int()
        ids[:, Skv // 4:Skv // 4 + 5] = -1
        kw["docs"] = ids.cuda()
    _attn_check(q, k, v, go, **kw)


@pytest.mark.parametrize("kind", ["none visible", "one token documents", "scattered", "rows"])
def test_attention_documents(kind):
    S = 300
    ids = {"none visible": torch.full((S,), -3), "one token documents": torch.arange(S), "scattered": torch.arange(S) * 7919 % 11,
           "rows": torch.where(torch.arange(S) % 3 == 0, -1, 2)}[kind].int()
    q, k, v, go = _attn_inputs(1, 4, 2, S, S, 64, torch.bfloat16, seed=2)
    docs = ids[None].cuda()
    out, lse, dq, dk, dv = _attn_check(q, k, v, go, docs=docs)
    if kind == "none visible":
        for t in (out, dq, dk, dv):
            assert (t == 0).all()
    if kind == "one token documents":
        assert torch.equal(out, v.repeat_interleave(2, 1))


@pytest.mark.parametrize("S, Sq, D", [(500, 500, 64), (300, 260, 128), (900, 1, 128)])
def test_attention_padding_may_hold_anything(S, Sq, D):
    q, k, v, go = _attn_inputs(2, 4, 2, Sq, S, D, torch.bfloat16, seed=3)
    ids = (torch.arange(S) // 97).int().repeat(2, 1)
    if Sq == 1:
        ids[:] = 3
    ids[0, 120:135] = -1
    ids[1, -40:-5] = -1
    docs, st = ids.cuda(), da.new_status()
    kw = dict(docs=docs, causal=True, softcap=30.0, status=st)

    def go_(q, k, v, g):
        out, lse = da.attention_forward(q, k, v, **kw)
        return (out, lse, *da.attention_backward(q, k, v, out, lse, g, **kw))
    a = go_(q, k, v, go)
    pad = docs < 0
    q, k, v, go = (t.clone() for t in (q, k, v, go))
    kp, qp = pad[:, None, :, None].expand_as(k), pad[:, None, S - Sq:, None].expand_as(q)
    for t, p, x in ((k, kp, float("nan")), (v, kp, float("inf")), (q, qp, float("nan")), (go, qp, float("-inf"))):
        t[p] = x
    for x, y in zip(a, go_(q, k, v, go)):
        assert torch.equal(x, y)
    assert da.read_status(st) == 0


def test_attention_padding_of_many_tiles():
    """Each tile holds padding, and tiles arrive in any order: their rows become zeros after they arrived, not before."""
    B, S = 8, 2600
    q, k, v, go = _attn_inputs(B, 16, 8, S, S, 128, torch.bfloat16, seed=6, heavy=False)
    ids = (torch.arange(S) // 500).int().repeat(B, 1)
    ids[:, ::50] = -1
    docs, st = ids.cuda(), da.new_status()
    for t in (q, k, v, go):
        t[:, :, ::50] = 0
    kw = dict(docs=docs, causal=True, status=st)
    out, lse = da.attention_forward(q, k, v, **kw)
    want = da.attention_backward(q, k, v, out, lse, go, **kw)
    for t in (q, k, v, go):
        t[:, :, ::50] = float("nan")
    for _ in range(10):
        o, l = da.attention_forward(q, k, v, **kw)
        assert torch.equal(o, out) and torch.equal(l, lse)
        for x, y in zip(da.attention_backward(q, k, v, o, l, go, **kw), want):
            assert torch.equal(x, y)
    assert da.read_status(st) == 0


@pytest.mark.parametrize("layout", ["bshd", "wide", "odd", "last"])
def test_attention_layouts(layout):
    q, k, v, go = _attn_inputs(2, 4, 2, 200, 200, 64, torch.bfloat16, seed=4, layout=layout)
    got = _attn_check(q, k, v, go, causal=True)
    want = [da.attention_forward(*(t.contiguous() for t in (q, k, v)), causal=True)[0]]
    assert torch.equal(got[0], want[0])
    if layout == "bshd":
        assert got[0].stride() == q.stride() and got[3].stride() == k.stride()


def test_attention_broadcast_and_autograd():
    """Expanded keys, a gradient that is an expanded view, and the autograd function against the calls."""
    q, k, v, go = _attn_inputs(2, 4, 1, 150, 150, 64, torch.bfloat16, seed=5)
    k1 = k[:1].clone().requires_grad_(True)
    q.requires_grad_(True)
    v.requires_grad_(True)
    out = da.attention(q, k1.expand(2, 1, 150, 64), v, causal=True, softcap=10.0)
    g1 = go[:, :, :1].expand_as(go)
    out.backward(g1)
    with torch.no_grad():
        kk = k1.expand(2, 1, 150, 64)
        o, lse = da.attention_forward(q, kk, v, causal=True, softcap=10.0)
        dq, dk, dv = da.attention_backward(q, kk, v, o, lse, g1.contiguous(), causal=True, softcap=10.0)
    assert torch.equal(o, out) and torch.equal(q.grad, dq) and torch.equal(v.grad, dv)
    assert torch.equal(k1.grad, dk.sum(0, keepdim=True))
    with torch.no_grad():
        assert torch.equal(da.attention(q, kk, v, causal=True, softcap=10.0), o)


def test_attention_scales():
    q, k, v, go = _attn_inputs(1, 2, 2, 140, 140, 64, torch.bfloat16, seed=6)
    for scale in (0.0, -0.1, 0.5):
        _attn_check(q, k, v, go, causal=True, scale=scale)
        _attn_check(q, k, v, go, causal=True, scale=scale, softcap=5.0)


def test_attention_moving_maximum():
    """Scores that grow from tile to tile by far more than the maximum's slack, and ones that fall."""
    q = torch.ones(1, 1, 200, 64, device="cuda", dtype=torch.bfloat16)
    for up in (True, False):
        ramp = torch.arange(640, device="cuda") / 8
        ramp = ramp if up else ramp.flip(0)
        k = (ramp[:, None] / 64).expand(640, 64).to(torch.bfloat16)[None, None].contiguous()
        g = torch.Generator(device="cuda").manual_seed(1)
        v = torch.randn(1, 1, 640, 64, device="cuda", generator=g).to(torch.bfloat16)
        go = torch.randn(1, 1, 200, 64, device="cuda", generator=g).to(torch.bfloat16)
        _attn_check(q, k, v, go, scale=1.0)
        _attn_check(q[:, :, :1], k, v, go[:, :, :1], scale=1.0)


def test_attention_gradient_agrees_with_differences():
    """f(x + h d) - f(x - h d) with x +- h d exact in f16: 2 h <grad, d> up to h^3 (h = 2^-6 on values of
    order 1: 2^-12 of the terms) and the roundings of the outputs, independent, u sqrt(2 sum (o g)^2)."""
    g = torch.Generator().manual_seed(7)
    q, k, v, go = ((torch.randint(-32, 33, (1, 2, 96, 64), generator=g) / 32).half().cuda() for _ in range(4))
    kw = dict(causal=True, softcap=8.0, slopes=torch.tensor([0.1, 0.0], device="cuda"))
    out, lse = da.attention_forward(q, k, v, **kw)
    grads = da.attention_backward(q, k, v, out, lse, go, **kw)
    h = 2.0 ** -6
    for i in range(3):
        d = torch.sign(grads[i])

        def f(s):
            x = [q, k, v]
            x[i] = (x[i].float() + s * h * d.float()).half()
            return (da.attention_forward(*x, **kw)[0].double() * go.double()).sum()
        slope = (f(1) - f(-1)) / (2 * h)
        want = grads[i].double().abs().sum()
        noise = 8 * 2.0 ** -11 * (2 * (out.double() * go.double()).square().sum()).sqrt() / (2 * h)
        assert abs(slope - want) <= 2.0 ** -9 * want + noise, i


def test_attention_same_bytes_on_another_stream_and_in_a_graph():
    q, k, v, go = _attn_inputs(2, 4, 2, 333, 333, 128, torch.bfloat16, seed=8)
    kw = dict(causal=True, softcap=30.0)
    xs = torch.randn(64, 512, device="cuda")
    w = torch.ones(512, device="cuda")

    def work():
        out, lse = da.attention_forward(q, k, v, **kw)
        y, mean, rstd = da.layer_norm_forward(xs, w, w)
        return [out, lse, *da.attention_backward(q, k, v, out, lse, go, **kw), y, *da.layer_norm_backward(xs, xs, w, mean, rstd)]
    a = work()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = work()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = work()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_attention_rows_do_not_depend_on_the_batch():
    q, k, v, go = _attn_inputs(3, 4, 2, 260, 260, 64, torch.bfloat16, seed=9)
    out, lse = da.attention_forward(q, k, v, causal=True)
    o1, l1 = da.attention_forward(q[1:2], k[1:2], v[1:2], causal=True)
    assert torch.equal(out[1:2], o1) and torch.equal(lse[1:2], l1)


@pytest.mark.parametrize("B, Hq, Hkv, Sq, S, D, dtype", [(16, 32, 8, 1, 4096, 128, torch.bfloat16), (19, 32, 8, 2, 2000, 64, torch.float16),
                                                         (40, 16, 16, 1, 1500, 128, torch.bfloat16), (64, 8, 8, 5, 700, 72, torch.bfloat16)])
def test_attention_many_requests_of_few_queries(B, Hq, Hkv, Sq, S, D, dtype):
    """More CTAs than SMs, each reading a cache of its own from memory: tiles arrive in any order, nothing may depend on it."""
    q, k, v, go = _attn_inputs(B, Hq, Hkv, Sq, S, D, dtype, seed=B, heavy=False)
    st = da.new_status()
    out, lse = da.attention_forward(q, k, v, causal=True, status=st)
    assert da.read_status(st) == 0
    for _ in range(40):
        again = da.attention_forward(q, k, v, causal=True, status=st)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert da.read_status(st) == 0
    b = slice(B - 2, B)
    r = R.attention(q[b], k[b], v[b], go[b], causal=True)
    _close(out[b], r["out"], R.attention_tolerance(r, dtype)["out"], "out")


def test_attention_empty():
    for B, Sq, Skv in ((0, 5, 5), (1, 0, 0), (1, 0, 7)):
        q = torch.zeros(B, 2, Sq, 64, device="cuda", dtype=torch.bfloat16)
        k = torch.zeros(B, 2, Skv, 64, device="cuda", dtype=torch.bfloat16)
        out, lse = da.attention_forward(q, k, k)
        dq, dk, dv = da.attention_backward(q, k, k, out, lse, q)
        assert out.shape == q.shape and (dk == 0).all() and (dv == 0).all()


def test_attention_offsets_past_32_bits():
    B, H, S = 9, 8, 262144                       # 4.8 GB of keys: element and byte offsets past 2^32
    k = torch.zeros(B, H, S, 128, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros(B, H, S, 128, device="cuda", dtype=torch.bfloat16)
    g = torch.Generator(device="cuda").manual_seed(2)
    k[-1, -1] = torch.randn(S, 128, device="cuda", generator=g).to(torch.bfloat16)
    v[-1, -1] = torch.randn(S, 128, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(B, H, 1, 128, device="cuda", generator=g).to(torch.bfloat16)
    out, lse = da.attention_forward(q, k, v)
    r = R.attention(q[-1:, -1:], k[-1:, -1:], v[-1:, -1:], q[-1:, -1:])
    _close(out[-1:, -1:], r["out"], R.attention_tolerance(r, torch.bfloat16)["out"] + 2.0 ** -13 * r["abs"]["out"], "out")
    assert (out[:-1] == 0).all()


# ---------------------------------------------------------------- layer norm

@pytest.mark.parametrize("dtype, wdtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                           (torch.bfloat16, torch.float32), (torch.float16, torch.float16)])
@pytest.mark.parametrize("rows, cols, gap", [(1, 1, 0), (3, 2, 0), (5, 31, 1), (70, 128, 0), (130, 257, 7), (9, 1000, 0), (700, 1024, 0),
                                             (33, 1030, 2), (40, 2048, 0), (21, 3001, 0), (650, 4096, 8), (12, 8200, 0), (5, 16384, 0),
                                             (7, 20000, 0), (3, 40001, 3)])
def test_layer_norm(rows, cols, gap, dtype, wdtype):
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x = (torch.randn(rows, cols + gap, device="cuda", generator=g) * 3 + 1).to(dtype)[:, :cols]
    dy = torch.randn(rows, cols + gap, device="cuda", generator=g).to(dtype)[:, :cols]
    w = (1 + 0.3 * torch.randn(cols, device="cuda", generator=g)).to(wdtype)
    b = (0.3 * torch.randn(cols, device="cuda", generator=g)).to(wdtype)
    y, mean, rstd = da.layer_norm_forward(x, w, b)
    dx, dw, db = da.layer_norm_backward(dy, x, w, mean, rstd)
    r = R.layer_norm(x, w, b, dy)
    tol = R.layer_norm_tolerance(r, dtype, wdtype, rows, cols)
    for got, n in ((y, "y"), (dx, "dx"), (dw, "dw"), (db, "db")):
        _close(got, r[n], tol[n], n)
    again = da.layer_norm_backward(dy, x, w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.parametrize("dtype, wdtype", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.float16, torch.float16)])
@pytest.mark.parametrize("rows, cols, gap", [(1300, 1100, 0), (1230, 2048, 0), (1250, 4096, 8), (1217, 8192, 0), (400, 1100, 4), (310, 2501, 3),
                                             (307, 1501, 0), (305, 6001, 0), (333, 8190, 2), (1, 5003, 0)])
def test_layer_norm_many_rows(rows, cols, gap, dtype, wdtype):
    """The streaming and the staged variants, which take many rows, with a last run that is shorter."""
    test_layer_norm(rows, cols, gap, dtype, wdtype)


def test_layer_norm_without_weights_and_shapes():
    x = torch.randn(4, 6, 50, device="cuda")
    y = da.layer_norm(x)
    r = R.layer_norm(x, None, None, x)
    _close(y, r["y"], 1e-5 * (1 + r["y"].abs()), "y")
    t = x.transpose(0, 1)                       # rows in no single stride
    assert torch.equal(da.layer_norm(t), y.transpose(0, 1))
    assert torch.equal(da.layer_norm(x[:, :, ::2]), da.layer_norm(x[:, :, ::2].contiguous()))
    assert da.layer_norm(x[:0]).shape == (0, 6, 50)
    assert torch.equal(da.layer_norm(x[1, 2]), y[1, 2])
    e = x[:, :1].expand(4, 6, 50)
    assert torch.equal(da.layer_norm(e), y[:, :1].expand(4, 6, 50))
    zero = da.layer_norm_backward(x[:0], x[:0], torch.ones(50, device="cuda"), *(torch.empty(0, 6, device="cuda"),) * 2)
    assert (zero[1] == 0).all() and (zero[2] == 0).all()


def test_layer_norm_constant_rows():
    x = torch.full((3, 100), 7.0, device="cuda")
    y, mean, rstd = da.layer_norm_forward(x, eps=1e-5)
    assert (y == 0).all() and (mean == 7).all()
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5))


def test_layer_norm_autograd_and_differences():
    """Central differences in f32 of sum(y g): 2^-24 of the terms over 2 h, and h^2 of curvature."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w, b, dy = (torch.randn(*s, device="cuda", generator=g) for s in ((40, 200), (200,), (200,), (40, 200)))
    for t in (x, w, b):
        t.requires_grad_(True)
    y = da.layer_norm(x, w, b)
    y.backward(dy)
    with torch.no_grad():
        for i, t in enumerate((x, w, b)):
            d, h = torch.sign(t.grad), 2.0 ** -7

            def f(s):
                a = [x, w, b]
                a[i] = a[i] + s * h * d
                return (da.layer_norm(*a).double() * dy.double()).sum()
            slope, want = (f(1) - f(-1)) / (2 * h), t.grad.double().abs().sum()
            assert abs(slope - want) <= 1e-3 * want
    only = torch.autograd.grad(da.layer_norm(x, w, None).sum(), w)[0]
    assert only.shape == w.shape


def test_layer_norm_offsets_past_32_bits():
    x = torch.zeros(70000, 32768, device="cuda", dtype=torch.bfloat16)
    x[-1] = torch.arange(32768, device="cuda").to(torch.bfloat16)
    y, mean, rstd = da.layer_norm_forward(x)
    r = R.layer_norm(x[-1:], None, None, x[-1:])
    _close(y[-1:], r["y"], R.layer_norm_tolerance(r, torch.bfloat16, torch.bfloat16, 1, 32768)["y"], "y")
    assert (y[:-1] == 0).all()


# ---------------------------------------------------------------- AdamW

def _adamw_plain(p, g, m, v, h, step, gs=None):
    """The documented operations on numpy's binary32, one rounding each."""
    f = np.float32
    b1, b2 = h["betas"]
    if gs is not None:
        g = g * f(gs)
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    root = np.sqrt(v)
    keep, rate, undo = f(1 - h["lr"] * h["weight_decay"]), f(h["lr"] / (1 - b1 ** step)), f(1 / np.sqrt(1 - b2 ** step))
    return p * keep - (m / (root * undo + f(h["eps"]))) * rate, m, v, root


H = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
SIZES = [1, 3, 255, 256, 257, 2048, 2049, 10001, 4]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("off", [0, 1])
def test_adamw_f32_states(dtype, off):
    g = torch.Generator().manual_seed(1)
    ps = [torch.randn(n + off, generator=g).to(dtype).cuda()[off:] for n in SIZES]     # off: starts that are not aligned
    m, v = (torch.zeros(da.adamw_state_len(ps), device="cuda") for _ in range(2))
    m.uniform_(-1e-3, 1e-3)
    pm, pv = m.cpu().numpy().copy(), v.cpu().numpy().copy()
    gs = torch.tensor([0.25], device="cuda")
    for step in (1, 2, 3):
        gr = [torch.randn(n + off, generator=g).to(dtype).cuda()[off:] for n in SIZES]
        gr[3] = None                                                                    # no gradient: nothing moves
        scale = gs if step == 3 else None
        want = [p.float().cpu().numpy() for p in ps]
        at = 0
        for i, n in enumerate(SIZES):
            if gr[i] is not None:
                s = slice(at, at + n)
                want[i], pm[s], pv[s], _ = _adamw_plain(want[i], gr[i].float().cpu().numpy(), pm[s], pv[s], H, step,
                                                        0.25 if step == 3 else None)
            at += -(-n // 256) * 256
        da.adamw_step(ps, gr, m, v, step, grad_scale=scale, **H)
        for p, w in zip(ps, want):
            assert torch.equal(p.cpu(), torch.from_numpy(w).to(dtype))
        assert np.array_equal(m.cpu().numpy(), pm) and np.array_equal(v.cpu().numpy(), pv)


def _pack8(x, positive):
    f = np.float32
    x = x.reshape(-1, 256)
    top = np.abs(x).max(1)
    live = top >= f(2.0 ** -100)
    scale = np.where(live, top / f(448), f(0)).astype(f)
    back = np.where(live, f(448) / np.where(live, top, f(1)), f(0)).astype(f)
    c = x * back[:, None]
    if positive:
        c = np.where((c > 0) & (c < f(2.0 ** -9)), f(2.0 ** -9), c)
    return torch.from_numpy(np.minimum(np.maximum(c, f(-448)), f(448))).to(torch.float8_e4m3fn).reshape(-1), scale


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_adamw_8bit_states(dtype):
    g = torch.Generator().manual_seed(2)
    ps = [torch.randn(n, generator=g).to(dtype).cuda() for n in SIZES]
    opt = da.AdamW(ps, state_bits=8, **H)
    s = opt.groups[0]
    n = s["exp_avg"].numel()
    m8, v8 = (torch.zeros(n).to(torch.float8_e4m3fn) for _ in range(2))
    ms, vs = np.zeros(n // 256, np.float32), np.zeros(n // 256, np.float32)
    for step in (1, 2, 3, 4):
        for p in ps:
            # magnitudes over twelve decades in one block: roots that would round to zero
            p.grad = (torch.randn(p.shape, generator=g) * 10.0 ** (-12 * torch.rand(p.shape, generator=g))).to(dtype).cuda()
            if step == 2:
                p.grad.zero_()
        m = m8.float().numpy() * np.repeat(ms, 256)
        r = v8.float().numpy() * np.repeat(vs, 256)
        want, m1, r1, at = [], np.zeros(n, np.float32), np.zeros(n, np.float32), 0
        for p in ps:
            k = slice(at, at + p.numel())
            w, m1[k], _, r1[k] = _adamw_plain(p.float().cpu().numpy(), p.grad.float().cpu().numpy(), m[k], r[k] * r[k], H, step)
            want.append(w)
            at += -(-p.numel() // 256) * 256
        m8, ms = _pack8(m1, False)
        v8, vs = _pack8(r1, True)
        opt.step()
        for p, w in zip(ps, want):
            assert torch.equal(p.cpu(), torch.from_numpy(w).to(dtype))
        assert np.array_equal(s["exp_avg_scale"].cpu().numpy(), ms) and np.array_equal(s["exp_avg_sq_scale"].cpu().numpy(), vs)
        assert torch.equal(s["exp_avg"].cpu().view(torch.uint8), m8.view(torch.uint8))
        assert torch.equal(s["exp_avg_sq"].cpu().view(torch.uint8), v8.view(torch.uint8))
        assert ((v8.float() > 0) == (torch.from_numpy(r1) > 0)).all() or (vs == 0).any()


def test_adamw_many_tensors_and_graph():
    """More tensors than one launch holds, mixed dtypes through the class, and a captured step."""
    g = torch.Generator().manual_seed(3)
    ps = [torch.randn(1 + 7 * i, generator=g).to(torch.bfloat16 if i % 2 else torch.float32).cuda() for i in range(300)]
    gr = [torch.randn(p.shape, generator=g).to(p.dtype).cuda() for p in ps]
    want = []
    for p, q in zip(ps, gr):
        z = np.zeros(p.numel(), np.float32)
        want.append(torch.from_numpy(_adamw_plain(p.float().cpu().numpy(), q.float().cpu().numpy(), z, z, H, 1)[0]).to(p.dtype))
    opt = da.AdamW(ps, **H)
    for p, q in zip(ps, gr):
        p.grad = q
    opt.step()
    assert all(torch.equal(p.cpu(), w) for p, w in zip(ps, want))
    p = torch.ones(5000, device="cuda")
    q = torch.full((5000,), 0.5, device="cuda")
    m, v = torch.zeros(2, 5120, device="cuda").unbind(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        da.adamw_step([p], [q], m, v, 1, **H)
    graph.replay()
    torch.cuda.synchronize()
    one = _adamw_plain(*(np.float32([x]) for x in (1, 0.5, 0, 0)), H, 1)[0]
    assert (p.cpu().numpy() == one).all()


def test_adamw_offsets_past_32_bits():
    n = 2 ** 31 + 5000
    p = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    q = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    p[-3:], q[-3:] = 1.0, 0.5
    k = da.adamw_state_len([p])
    m, v = (torch.zeros(k, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ms, vs = torch.zeros(2, k // 256, device="cuda").unbind(0)
    da.adamw_step([p], [q], m, v, 1, exp_avg_scale=ms, exp_avg_sq_scale=vs, **H)
    one = torch.from_numpy(_adamw_plain(*(np.float32([x]) for x in (1, 0.5, 0, 0)), H, 1)[0]).to(torch.bfloat16)
    assert (p[-3:].cpu() == one).all() and (p[:-3] == 0).all()
    assert (ms[:-1] == 0).all() and ms[-1] > 0
