"""Host-side checks of the training operators: the C ABI refuses bad arguments before any launch,
the binding refuses bad tensors before the library, and the 64-bit references of the GPU tests have
gradients that agree with differences."""
import ctypes as C
import math
import os
import sys

import pytest
import torch

import bitwise_deterministic_shard_gb300 as da
from bitwise_deterministic_shard_gb300 import train

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import train_reference as R  # noqa: E402


@pytest.fixture(scope="module")
def L():
    from bitwise_deterministic_shard_gb300 import build
    build.build()
    return da.lib()


def _desc(B=1, Hq=4, Hkv=2, Sq=8, Skv=8, D=64, dtype=1):
    d = train._Train()
    for t, H, S in ((d.q, Hq, Sq), (d.k, Hkv, Skv), (d.v, Hkv, Skv)):
        t.ptr, t.dtype, t.B, t.H, t.S, t.D = 4096, dtype, B, H, S, D
        t.stride[:] = (H * S * D, S * D, D, 1)
    d.scale = math.nan
    return d


def _refuse(change):
    d = _desc()
    change(d)
    return d


@pytest.mark.parametrize("change, code", [
    (lambda d: setattr(d.q, "dtype", 0), 3),                       # f32
    (lambda d: setattr(d.v, "dtype", 2), 3),                       # mixed
    (lambda d: setattr(d.k, "H", 3), 2),                           # Hq % Hkv
    (lambda d: setattr(d.q, "S", 9), 2),                           # Sq > Skv
    (lambda d: [setattr(t, "D", 60) for t in (d.q, d.k, d.v)], 2),  # D % 8
    (lambda d: [setattr(t, "D", 136) for t in (d.q, d.k, d.v)], 2),  # D > 128
    (lambda d: setattr(d.q, "ptr", 4104), 4),                      # 16-byte alignment
    (lambda d: d.q.stride.__setitem__(2, 68), 4),                  # a stride off 16 bytes
    (lambda d: d.k.stride.__setitem__(1, 0), 2),                   # broadcast heads
    (lambda d: d.q.stride.__setitem__(3, 2), 2),
    (lambda d: setattr(d.k, "ptr", None), 1),
    (lambda d: setattr(d, "softcap", -1.0), 1),
    (lambda d: setattr(d, "softcap", math.nan), 1),
    (lambda d: setattr(d, "softcap", math.inf), 1),
    (lambda d: setattr(d, "scale", math.inf), 1),
    (lambda d: setattr(d, "prefix", 4096), 1),                     # prefix without causal
    (lambda d: setattr(d, "docs", 4098), 4),
    (lambda d: setattr(d, "slopes", 4098), 4),
])
def test_attention_descriptor_is_refused(L, change, code):
    d = _refuse(change)
    assert L.dta_workspace_bytes(C.byref(d), 0) == 0 and L.dta_workspace_bytes(C.byref(d), 1) == 0
    assert L.dta_forward(C.byref(d), C.byref(d.q), None, None, 0, None) == code
    o = _desc()
    assert L.dta_backward(C.byref(d), C.byref(o.q), 4096, C.byref(o.q), C.byref(o.q), C.byref(o.k), C.byref(o.v), 4096, 0, None) == code


def test_attention_outputs_and_workspace_are_checked(L):
    d, o = _desc(), _desc()
    assert L.dta_forward(None, C.byref(o.q), None, None, 0, None) == 1
    assert L.dta_forward(C.byref(d), None, None, None, 0, None) == 1
    assert L.dta_forward(C.byref(d), C.byref(o.k), None, None, 0, None) == 2              # shaped as k
    o.q.dtype = 2
    assert L.dta_forward(C.byref(d), C.byref(o.q), None, None, 0, None) == 3
    o = _desc()
    assert L.dta_forward(C.byref(d), C.byref(o.q), 4098, None, 0, None) == 4
    need = L.dta_workspace_bytes(C.byref(d), 1)
    assert need >= 4 * 128 * 8
    back = lambda lse, ws, n: L.dta_backward(C.byref(d), C.byref(o.q), lse, C.byref(o.q), C.byref(o.q), C.byref(o.k),  # noqa: E731
                                             C.byref(o.v), ws, n, None)
    assert back(None, 4096, need) == 1
    assert back(4096, None, 0) == 5 and back(4096, 4096, need - 1) == 5
    assert back(4096, 4096 + 128, need) == 4


def test_workspace_of_the_split_forward_is_bounded(L):
    """The key ranges of the few-query form never exceed what the SMs can take at once."""
    for B in (1, 8, 64, 500):
        for Skv in (1, 127, 512, 8192, 131072):
            d = _desc(B=B, Hq=8, Hkv=2, Sq=1, Skv=Skv, D=128)
            n = L.dta_workspace_bytes(C.byref(d), 0)
            if Skv <= 512:                       # up to four tiles are not worth a join
                assert n == 0
            else:
                assert (B > 8 or n > 0) and n <= 2 * 64 * B * 2 * 128 * 130 * 4 + 512     # many requests: no split, no sums


def _matrix(rows=4, cols=10, dtype=0, stride=None, ptr=4096):
    m = da._Matrix()
    m.ptr, m.dtype, m.rows, m.cols, m.row_stride = ptr, dtype, rows, cols, cols if stride is None else stride
    return m


@pytest.mark.parametrize("x, y, wdtype, w, eps, mean, code", [
    (_matrix(), _matrix(dtype=1), 0, 4096, 1e-5, 4096, 3),
    (_matrix(dtype=1), _matrix(dtype=1), 2, 4096, 1e-5, 4096, 3),
    (_matrix(dtype=7), _matrix(dtype=7), 0, 4096, 1e-5, 4096, 3),
    (_matrix(stride=9), _matrix(), 0, 4096, 1e-5, 4096, 2),
    (_matrix(), _matrix(rows=5), 0, 4096, 1e-5, 4096, 2),
    (_matrix(cols=0, stride=0), _matrix(cols=0, stride=0), 0, 4096, 1e-5, 4096, 2),
    (_matrix(ptr=None), _matrix(), 0, 4096, 1e-5, 4096, 1),
    (_matrix(ptr=4098), _matrix(), 0, 4096, 1e-5, 4096, 4),
    (_matrix(), _matrix(), 0, 4098, 1e-5, 4096, 4),
    (_matrix(), _matrix(), 0, 4096, -1.0, 4096, 1),
    (_matrix(), _matrix(), 0, 4096, math.nan, 4096, 1),
    (_matrix(), _matrix(), 0, 4096, 1e-5, None, 1),
    (_matrix(), _matrix(), 0, 4096, 1e-5, 4098, 4),
])
def test_layer_norm_forward_is_refused(L, x, y, wdtype, w, eps, mean, code):
    assert L.dln_forward(C.byref(x), w, None, wdtype, eps, C.byref(y), mean, 4096, None) == code


def test_layer_norm_backward_is_refused(L):
    x, ok = _matrix(), 4096
    call = lambda dy, dw, ws, n, mean=ok: L.dln_backward(C.byref(dy), C.byref(x), ok, 0, mean, ok, C.byref(_matrix()),  # noqa: E731
                                                        dw, None, ws, n, None)
    assert call(_matrix(rows=3), None, None, 0) == 2
    assert call(_matrix(dtype=1), None, None, 0) == 3
    assert call(_matrix(), ok, None, 0) == 5
    assert call(_matrix(), ok, ok + 4, L.dln_workspace_bytes(4, 10)) == 4
    assert call(_matrix(), None, None, 0, mean=None) == 1
    assert L.dln_workspace_bytes(-1, 10) == 0 and L.dln_workspace_bytes(4, 0) == 0


def test_adamw_is_refused(L):
    h = train._Hyper(1e-3, 0.9, 0.99, 1e-8, 0.0, 1)
    t = (train._Param * 1)(train._Param(4096, 4096, 100, 0))

    def call(n=1, dtype=0, bits=32, m=4096, scale=None, length=256, hyper=h):
        return L.dow_adamw(t, n, dtype, bits, m, m, scale, scale, length, C.byref(hyper), None, None)
    assert L.dow_adamw(t, 1, 0, 32, 4096, 4096, None, None, 256, None, None, None) == 1
    assert call(n=-1) == 1 and call(dtype=5) == 3 and call(bits=16) == 1 and call(m=None) == 1
    assert call(bits=8) == 1                                          # no scales
    assert call(length=200) == 2 and call(length=0) == 2
    assert call(m=4100) == 4
    for bad in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(step=0), dict(lr=math.inf), dict(eps=math.nan)):
        kw = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, **{})
        kw.update(bad)
        assert call(hyper=train._Hyper(*[kw[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay", "step")])) == 1
    for field, value, code in (("state", 100, 2), ("state", 256, 2), ("numel", 257, 2), ("numel", -1, 2), ("param", None, 1),
                               ("grad", 4098, 4)):
        keep = getattr(t[0], field)
        setattr(t[0], field, value)
        assert call() == code, field
        setattr(t[0], field, keep)
    t[0].numel = 0
    assert call(m=None) == 0                                          # nothing to do


class _Nothing:
    def __getattr__(self, name):
        raise AssertionError(f"the library was reached: {name}")


@pytest.fixture
def nolib(monkeypatch):
    monkeypatch.setattr(da, "_cuda", lambda t, name: None)
    monkeypatch.setattr(da, "lib", lambda: _Nothing())


def _qkv(dtype=torch.bfloat16, D=64, S=8):
    return torch.zeros(1, 4, S, D, dtype=dtype), torch.zeros(1, 2, S, D, dtype=dtype), torch.zeros(1, 2, S, D, dtype=dtype)


@pytest.mark.parametrize("kw", [
    dict(slopes=torch.zeros(3)), dict(slopes=torch.zeros(4, dtype=torch.float64)), dict(slopes=torch.zeros(4, requires_grad=True)),
    dict(docs=torch.zeros(1, 8, dtype=torch.int64)), dict(docs=torch.zeros(1, 9, dtype=torch.int32)),
    dict(prefix=torch.zeros(2, dtype=torch.int32)), dict(prefix=torch.zeros(1))])
def test_binding_refuses_attention_options(nolib, kw):
    with pytest.raises(da.DetAttnError):
        da.attention(*_qkv(), **kw)


def test_binding_refuses_attention_tensors(nolib):
    q, k, v = _qkv()
    for bad in ((q.float(), k.float(), v.float()), (q, k.half(), v), (q[0], k, v)):
        with pytest.raises(da.DetAttnError):
            da.attention(*bad)
    with pytest.raises(da.DetAttnError):
        da.attention_backward(q, k, v, q, torch.zeros(1, 4, 7), q)
    with pytest.raises(da.DetAttnError):
        da.attention_backward(q, k, v, q, torch.zeros(1, 4, 8), q.float())
    with pytest.raises(da.DetAttnError):
        da.attention_forward(q, k, v, out=torch.zeros(1, 4, 8, 64))


def test_binding_refuses_layer_norm_tensors(nolib):
    x = torch.zeros(4, 10)
    for args in ((x.double(),), (x, torch.ones(9)), (x, torch.ones(10).bfloat16()), (x, torch.ones(10), torch.ones(10).half()),
                 (torch.zeros(4, 0),), (torch.zeros(()),)):
        with pytest.raises(da.DetAttnError):
            da.layer_norm(*args)
    s = torch.zeros(4)
    for args in ((x.half(), x, None, s, s), (x, x, None, torch.zeros(3), s), (x, x, None, s, s.double()), (x[:3], x, None, s, s)):
        with pytest.raises(da.DetAttnError):
            da.layer_norm_backward(*args)


def test_binding_refuses_adamw_tensors(nolib):
    p, m = [torch.zeros(10), torch.zeros(300)], torch.zeros(768)
    g = [torch.zeros(10), torch.zeros(300)]
    assert da.adamw_state_len(p) == 768
    for args, kw in ((([p[0]], g, m, m), {}), ((p, [g[0], g[1].half()], m, m), {}), ((p, [g[0], torch.zeros(299)], m, m), {}),
                     ((p, g, m[:512], m), {}), ((p, g, m, m.double()), {}), ((p, g, m, m), dict(exp_avg_scale=torch.zeros(3))),
                     (([p[0], p[1].half()], g, m, m), {}), ((p, g, m.to(torch.float8_e4m3fn), m.to(torch.float8_e4m3fn)), {}),
                     ((p, g, m, m), dict(grad_scale=torch.zeros(2))), (([p[0].double()], [g[0].double()], m[:256], m[:256]), {})):
        with pytest.raises(da.DetAttnError):
            da.adamw_step(*args, 1, **kw)
    with pytest.raises(da.DetAttnError):
        da.AdamW(p, state_bits=16)


@pytest.mark.parametrize("kw", [dict(causal=True, softcap=2.0), dict(slopes=True), dict(causal=True, prefix=True, docs=True)])
def test_reference_gradients_agree_with_differences(kw):
    """The references' formulas against central differences: h^2 curvature and 2^-53 / h rounding
    leave about 1e-9 of the values with h = 1e-5; 1e-7 is allowed."""
    g = torch.Generator().manual_seed(3)
    q, k, v, go = (torch.randn(2, h, 9, 8, generator=g, dtype=torch.float64) for h in (4, 2, 2, 4))
    kw = dict(kw)
    if kw.get("slopes"):
        kw["slopes"] = torch.tensor([0.5, 0.25, 0.1, 0.0])
    if kw.get("docs"):
        kw["docs"] = torch.tensor([[0, 0, 0, 1, 1, 1, 1, -1, -1], [5] * 9], dtype=torch.int32)
    if kw.get("prefix"):
        kw["prefix"] = torch.tensor([4, 0], dtype=torch.int32)
    r = R.attention(q, k, v, go, **kw)
    for x, name in ((q, "dq"), (k, "dk"), (v, "dv")):
        d = torch.randn(x.shape, generator=g, dtype=torch.float64)
        h, keep = 1e-5, x.clone()
        x += h * d
        up = (R.attention(q, k, v, go, **kw)["out"] * go).sum()
        x.copy_(keep - h * d)
        down = (R.attention(q, k, v, go, **kw)["out"] * go).sum()
        x.copy_(keep)
        assert abs((up - down) / (2 * h) - (r[name] * d).sum()) < 1e-7 * (1 + r[name].abs().sum())
    x, w, b, dy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((5, 7), (7,), (7,), (5, 7)))
    r = R.layer_norm(x, w, b, dy)
    for t, name in ((x, "dx"), (w, "dw"), (b, "db")):
        d, keep = torch.randn(t.shape, generator=g, dtype=torch.float64), t.clone()
        t += 1e-5 * d
        up = (R.layer_norm(x, w, b, dy)["y"] * dy).sum()
        t.copy_(keep - 1e-5 * d)
        down = (R.layer_norm(x, w, b, dy)["y"] * dy).sum()
        t.copy_(keep)
        assert abs((up - down) / 2e-5 - (r[name] * d).sum()) < 1e-7 * (1 + r[name].abs().sum())


def test_references_reject_planted_mistakes():
    """A mistake planted in a reference moves it by more than the GPU tests' tolerances."""
    g = torch.Generator().manual_seed(4)
    q, k, v, go = (torch.randn(1, 2, 40, 16, generator=g, dtype=torch.float64) for _ in range(4))
    kw = dict(causal=True, softcap=3.0, slopes=torch.tensor([0.3, 0.1]))
    r = R.attention(q, k, v, go, **kw)
    tol = R.attention_tolerance(r, torch.bfloat16)
    for wrong in (dict(causal=False), dict(softcap=4.0), dict(softcap=0.0), dict(slopes=-kw["slopes"]), dict(scale=0.3)):
        w = R.attention(q, k, v, go, **{**kw, **wrong})
        assert all((w[n] - r[n] > tol[n]).any() for n in ("out", "dq", "dk", "dv")), wrong
    x, w_, b, dy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((50, 32), (32,), (32,), (50, 32)))
    r, wrong = R.layer_norm(x, w_, b, dy), R.layer_norm(x, w_, b, dy, eps=1e-2)
    tol = R.layer_norm_tolerance(r, torch.bfloat16, torch.float32, 50, 32)
    assert ((wrong["dw"] - r["dw"]).abs() > tol["dw"]).any()
