"""Host-side checks of the decoder's operators: the C ABI refuses bad arguments before any launch, the binding refuses bad tensors
before the library, the 64-bit references of the GPU tests have gradients that agree with differences, and mistakes planted in
them are larger than the tolerances."""
import ctypes as C
import math
import os
import sys

import pytest
import torch

import bitwise_deterministic_shard_gb300 as da
from bitwise_deterministic_shard_gb300 import decoder, train

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import decoder_reference as R  # noqa: E402


@pytest.fixture(scope="module")
def L():
    from bitwise_deterministic_shard_gb300 import build
    build.build()
    return da.lib()


def M(rows=16, cols=64, dtype=1, stride=None, ptr=4096):
    m = da._Matrix()
    m.ptr, m.dtype, m.rows, m.cols, m.row_stride = ptr, dtype, rows, cols, cols if stride is None else stride
    return m


def ref(m):
    return None if m is None else C.byref(m)


# ---------------------------------------------------------------- C ABI

@pytest.mark.parametrize("x, wg, wu, act, h, saved, code", [
    (None, M(32), M(32), 0, M(16, 32), None, 1),
    (M(dtype=0), M(32, dtype=0), M(32, dtype=0), 0, M(16, 32, dtype=0), None, 3),
    (M(), M(32, dtype=2), M(32, dtype=2), 0, M(16, 32), None, 3),
    (M(), M(32), M(32, dtype=2), 0, M(16, 32), None, 3),
    (M(), M(32), M(40), 0, M(16, 32), None, 2),
    (M(), M(32, 72), M(32, 72), 0, M(16, 32), None, 2),
    (M(cols=60), M(32, 60), M(32, 60), 0, M(16, 32), None, 2),
    (M(), M(30), M(30), 0, M(16, 30), None, 2),
    (M(), M(32), M(32), 0, M(16, 40), None, 2),
    (M(), M(32), M(32), 0, M(15, 32), None, 2),
    (M(), M(32), M(32), 4, M(16, 32), None, 1),
    (M(), M(32), M(32), -1, M(16, 32), None, 1),
    (M(), M(32), M(32), 0, M(16, 32), 4104, 4),
    (M(stride=56), M(32), M(32), 0, M(16, 32), None, 2),
    (M(stride=68), M(32), M(32), 0, M(16, 32), None, 4),
    (M(ptr=4104), M(32), M(32), 0, M(16, 32), None, 4),
    (M(), M(32), M(32), 0, M(16, 32, ptr=4112 + 8), None, 4),
    (M(ptr=None), M(32), M(32), 0, M(16, 32), None, 1),
    (M(rows=1 << 25), M(32), M(32), 0, M(1 << 25, 32), None, 2)])
def test_gated_forward_is_refused(L, x, wg, wu, act, h, saved, code):
    assert L.dgl_forward(ref(x), ref(wg), ref(wu), act, ref(h), saved, None, None) == code


def test_gated_backward_is_refused(L):
    need = L.dgl_workspace_bytes(16, 32)
    assert need >= 4 * 16 * 32 and L.dgl_saved_bytes(16, 32) == 6 * 16 * 32 and L.dgl_saved_bytes(3, 40) == 6 * 3 * 48
    assert L.dgl_workspace_bytes(-1, 8) == 0 and L.dgl_saved_bytes(1, 1 << 25) == 0

    def call(dh=M(16, 32), x=M(), saved=4096, dx=M(), dwg=M(32), dwu=M(32), ws=4096, n=need, status=None):
        return L.dgl_backward(ref(dh), ref(x), ref(M(32)), ref(M(32)), saved, ref(dx), ref(dwg), ref(dwu), ws, n, status, None)
    assert call(dh=None) == 1 and call(dh=M(16, 40)) == 2 and call(dh=M(16, 32, dtype=2)) == 3
    assert call(dx=M(15)) == 2 and call(dx=M(dtype=2)) == 3 and call(dx=M(ptr=4100)) == 4
    assert call(dwg=None) == 1 and call(dwu=None) == 1 and call(dwg=M(40)) == 2
    assert call(saved=None) == 1 and call(saved=4104) == 4
    assert call(ws=None) == 5 and call(n=need - 1) == 5 and call(ws=4096 + 128) == 4
    assert call(status=4098) == 4
    assert call(dx=None, dwg=None, dwu=None) == 0                       # nothing is wanted


def test_log_probs_are_refused(L):
    ok = 4096

    def call(x=M(4, 100, 0), targets=ok, temperature=1.0, top=0, lp=ok, h=ok, saved=None, tlp=None, ti=None, status=None):
        return L.dlp_forward(ref(x), targets, temperature, top, lp, h, saved, tlp, ti, status, None)
    assert call(x=None) == 1 and call(x=M(4, 100, 7)) == 3 and call(x=M(4, 0, 0)) == 2 and call(x=M(4, 100, 0, 99)) == 2
    assert call(x=M(4, 100, 0, ptr=4098)) == 4 and call(x=M(4, 100, 0, ptr=None)) == 1
    for t in (0.0, -1.0, math.nan, math.inf, 2.0 ** 61, 2.0 ** -61):
        assert call(temperature=t) == 1
    assert call(top=-1) == 1 and call(top=33) == 1 and call(x=M(4, 5, 0), top=6) == 1 and call(top=3) == 1
    assert call(targets=None) == 1 and call(lp=None) == 1 and call(h=None) == 1
    assert call(targets=4100) == 4 and call(lp=4098) == 4 and call(saved=4098) == 4 and call(top=3, tlp=ok, ti=4100) == 4
    assert call(x=M(1 << 30, 1 << 20, 0)) == 2
    assert call(x=M(0, 100, 0), targets=None) == 0                      # no rows

    def back(x=M(4, 100, 0), targets=ok, saved=ok, g=None, h=None, temperature=1.0, dx=M(4, 100, 0)):
        return L.dlp_backward(ref(x), targets, saved, g, h, temperature, ref(dx), None)
    assert back(dx=None) == 1 and back(dx=M(4, 99, 0)) == 2 and back(dx=M(4, 100, 1)) == 3 and back(saved=None) == 1
    assert back(targets=None) == 1 and back(temperature=0.0) == 1 and back(g=4098) == 4 and back(h=4098) == 4
    assert back(x=M(0, 100, 0), dx=M(0, 100, 0), saved=None) == 0


def test_embedding_is_refused(L):
    ok = 4096

    def call(ids=ok, bits=64, w=M(50, 20, 0), scale=1.0, y=M(8, 20, 0), status=None):
        return L.dte_forward(ids, bits, ref(w), scale, ref(y), status, None)
    assert call(w=None) == 1 and call(y=None) == 1 and call(y=M(8, 20, 1)) == 3 and call(y=M(8, 21, 0)) == 2 and call(w=M(0, 20, 0)) == 2
    assert call(bits=16) == 1 and call(ids=None) == 1 and call(ids=4100) == 4 and call(bits=32, ids=4098) == 4
    assert call(scale=math.inf) == 1 and call(scale=math.nan) == 1 and call(status=4098) == 4
    assert call(ids=None, y=M(0, 20, 0)) == 0
    need = L.dte_workspace_bytes(8, 20)
    assert need > 0 and L.dte_workspace_bytes(-1, 5) == 0 and L.dte_workspace_bytes(5, 0) == 0

    def back(ids=ok, bits=64, dy=M(8, 20, 0), scale=1.0, padding=-1, dw=M(50, 20, 0), ws=ok, n=need, status=None):
        return L.dte_backward(ids, bits, ref(dy), scale, padding, ref(dw), ws, n, status, None)
    assert back(dy=M(8, 20, 1)) == 3 and back(dy=M(8, 19, 0)) == 2 and back(padding=50) == 1 and back(padding=-2) == 1
    assert back(ws=None) == 5 and back(n=need - 1) == 5 and back(ws=ok + 64) == 4 and back(scale=math.nan) == 1 and back(bits=8) == 1


def test_workspaces_hold_every_list(L):
    """The sorted places, a chunk each token at most, the sums of chunks."""
    for n in (1, 32, 33, 4096, 4097, 32768, 32769, 1 << 20):
        for cols in (1, 1000):
            b = L.dte_workspace_bytes(n, cols)
            sums = 8 * (n // 32 + 1) * cols if n > 32 else 0
            assert sums + 20 * n <= b <= sums + 20 * n + (12 * n + 2048 * (n // 1024 + 1) if n > 4096 else 0) + n + 4096


# ---------------------------------------------------------------- binding

class _Library:
    """Records the calls, succeeds, and does nothing."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 6 * a[0] * ((a[1] + 15) // 16 * 16) if name == "dgl_saved_bytes" else 4096
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def stub(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(da, "_cuda", lambda t, name: None)
    monkeypatch.setattr(da, "lib", lambda: lib)
    monkeypatch.setattr(decoder, "_on", lambda index, name, t: None)
    monkeypatch.setattr(train, "_on", lambda index, name, t: None)
    monkeypatch.setattr(decoder, "_run", lambda what, index, f, *args: f(*args) and None)
    return lib


B16 = torch.bfloat16


def test_binding_refuses_gated_tensors(stub):
    x, w = torch.zeros(4, 16, dtype=B16), torch.zeros(24, 16, dtype=B16)
    for args in ((x.float(), w.float(), w.float()), (x, w, w.half()), (x, w, w[:16]), (x, w[:, :8], w[:, :8]), (x, w[0], w[0]),
                 (x[:, :12], w[:, :12], w[:, :12]), (x, w[:20], w[:20]), (x, w, w, "swish")):
        with pytest.raises(da.DetAttnError):
            da.gated_linear(*args)
    with pytest.raises(da.DetAttnError):
        da.gated_linear_forward(x, w, w, out=torch.zeros(4, 16, dtype=B16))
    h, saved = da.gated_linear_forward(x, w, w)
    for bad in (h.half(), h[:3], h[:, :16]):
        with pytest.raises(da.DetAttnError):
            da.gated_linear_backward(bad, x, w, w, saved)
    for bad in (saved[:-1], saved.float()):
        with pytest.raises(da.DetAttnError):
            da.gated_linear_backward(h, x, w, w, bad)
    assert [c[0] for c in stub.calls] == ["dgl_forward"]


def test_binding_refuses_logits(stub):
    x, t = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int64)
    for args, kw in (((x.double(), t), {}), ((x, t[:3]), {}), ((x, t.float()), {}), ((x, t), dict(top=11)), ((x, t), dict(top=-1)),
                     ((torch.zeros(4, 50), t), dict(top=33)), ((x, t), dict(temperature=0.0)), ((x, t), dict(temperature=math.nan)),
                     ((x[:, :0], t), {}), ((x, t.bool()), {})):
        with pytest.raises(da.DetAttnError):
            da.log_probs(*args, **kw)
    _, saved = da.log_probs_forward(x, t)
    g = torch.zeros(4)
    for args, kw in (((x, t, saved[:3], g), {}), ((x, t, saved, g[:3]), {}), ((x, t, saved, g.double()), {}),
                     ((x, t, saved, g, g.half()), {}), ((x, t, saved, g), dict(out=torch.zeros(4, 9)))):
        with pytest.raises(da.DetAttnError):
            da.log_probs_backward(*args, **kw)


def test_binding_refuses_embedding_tensors(stub):
    w, ids = torch.zeros(10, 8), torch.zeros(5, dtype=torch.int64)
    for args, kw in (((ids.float(), w), {}), ((ids, w.double()), {}), ((ids, w[0]), {}), ((ids, w[:0]), {}), ((ids, w), dict(padding_idx=10)),
                     ((ids, w), dict(padding_idx=-1)), ((ids.short(), w), {})):
        with pytest.raises(da.DetAttnError):
            da.embedding(*args, **kw)
    for args, kw in (((torch.zeros(4, 8), ids, 10), {}), ((torch.zeros(5, 8), ids, 0), {}), ((torch.zeros(5, 8), ids, 10), dict(padding_idx=10)),
                     ((torch.zeros(5, 8).double(), ids, 10), {})):
        with pytest.raises(da.DetAttnError):
            da.embedding_backward(*args, **kw)
    with pytest.raises(da.DetAttnError):
        da.embedding_forward(ids, w, out=torch.zeros(5, 9))


def test_binding_refuses_a_missing_saved_tensor(stub):
    x, w, t = torch.zeros(4, 16, dtype=B16), torch.zeros(24, 16, dtype=B16), torch.zeros(4, dtype=torch.int64)
    h, saved = da.gated_linear_forward(x, w, w, need_saved=False)
    with pytest.raises(da.DetAttnError):
        da.gated_linear_backward(h, x, w, w, saved)
    _, saved = da.log_probs_forward(x, t, need_saved=False)
    with pytest.raises(da.DetAttnError):
        da.log_probs_backward(x, t, saved, torch.zeros(4))


def test_layouts_that_are_passed_on_and_copied(stub):
    """One run of rows goes to the kernels as it is, 16-byte rows apart where they are needed; others are copied."""
    big = torch.zeros(6, 5, 32, dtype=B16)
    for t, cols, run in ((big, 32, 32), (big[:, :, :24], 24, 32), (big[0], 32, 32), (big[:, 1], 32, 160), (big[::2], 32, None),
                         (big.transpose(0, 1), 32, None), (big[:1, :, :8], 8, 32), (big[0, 0], 32, 32), (big[:, :, ::2], 16, None),
                         (torch.zeros(1, 1, dtype=B16).expand(6, 32), 32, None), (big[:0], 32, 32)):
        assert decoder._run_of_rows(t, cols) == run
    w = torch.zeros(24, 24, dtype=B16)
    for x, copied in ((big[:, :, :24], False), (big[:, :, 4:28], True), (torch.zeros(4, 28, dtype=B16)[:, :24], True), (big[::2, :, :24], True)):
        da.gated_linear(x, w, w)
        at = train._MATRIX.unpack(stub.calls[-1][1][0])
        assert (at[0] != x.data_ptr()) == copied and at[0] % 16 == 0 and at[3] % 8 == 0


def test_gradients_have_their_tensors_layout(stub):
    x = torch.zeros(4, 40, dtype=torch.float16)[:, :35]
    t, g = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    _, saved = da.log_probs_forward(x, t)
    dx = da.log_probs_backward(x, t, saved, g)
    assert dx.shape == x.shape and dx.stride() == (40, 1)               # rows start on 16 bytes as the logits' do
    x = torch.zeros(4, 100)[:, :33]
    dx = da.log_probs_backward(x, t, da.log_probs_forward(x, t)[1], g)
    assert dx.stride() == (36, 1)
    x = torch.zeros(4, 33)
    assert da.log_probs_backward(x, t, saved, g).is_contiguous()


def test_autograd_of_the_operators(stub):
    """Each leaf gets a gradient of its shape and type, where it needs one; what has none gets none."""
    x, w, v = (torch.zeros(*s, dtype=B16, requires_grad=True) for s in ((2, 3, 16), (24, 16), (24, 16)))
    h = da.gated_linear(x, w, v, "gelu")
    h.sum().backward()
    assert h.shape == (2, 3, 24) and x.grad.shape == x.shape and w.grad.shape == w.shape and v.grad.dtype == B16
    da.gated_linear(x.detach(), w, v.detach()).sum().backward()
    assert stub.calls[-1][1][5] is None                                # no dx
    z = torch.zeros(4, 9, requires_grad=True)
    r = da.log_probs(z, torch.zeros(4, dtype=torch.int32), top=3)
    assert not r.top_log_probs.requires_grad and not r.top_indices.requires_grad and r.top_indices.dtype == torch.int64
    (r.log_probs.sum()).backward()
    assert z.grad.shape == z.shape and stub.calls[-1][1][4] is None     # no gradient of the entropy
    e = torch.zeros(7, 8, requires_grad=True)
    da.embedding(torch.zeros(2, 3, dtype=torch.int32), e, 2.0, padding_idx=1).sum().backward()
    assert e.grad.shape == e.shape and stub.calls[-1][1][4] == 1
    with torch.no_grad():
        assert not da.gated_linear(x, w, v).requires_grad and not da.embedding(torch.zeros(1, dtype=torch.int64), e).requires_grad
        assert not da.log_probs(z, torch.zeros(4, dtype=torch.int64)).log_probs.requires_grad


def test_tensors_may_not_change_before_the_backward_pass(stub):
    ids, t = torch.zeros(3, dtype=torch.int64), torch.zeros(4, dtype=torch.int64)
    z = torch.zeros(4, 9, requires_grad=True)
    e = torch.zeros(7, 8, requires_grad=True)
    for out, changed in ((da.embedding(ids, e), ids), (da.log_probs(z, t).log_probs, t)):
        out.sum().backward(retain_graph=True)
        changed.add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.sum().backward()


def test_writes_and_forward_mode(stub):
    x, w = torch.zeros(4, 16, dtype=B16), torch.zeros(24, 16, dtype=B16)
    outs = [torch.zeros(4, 24, dtype=B16), torch.zeros(3, 8), torch.zeros(4, 9)]
    da.gated_linear_forward(x, w, w, out=outs[0])
    da.embedding_forward(torch.zeros(3, dtype=torch.int64), torch.zeros(7, 8), out=outs[1])
    z, t = outs[2], torch.zeros(4, dtype=torch.int64)
    da.log_probs_backward(z, t, da.log_probs_forward(z, t)[1], torch.zeros(4), out=z)     # in place of the logits
    assert [o._version for o in outs] == [1, 1, 1]
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        dual = lambda a: fwd.make_dual(a, torch.ones_like(a))  # noqa: E731
        for f in (lambda: da.gated_linear(dual(x), w, w), lambda: da.gated_linear(x, w, dual(w)),
                  lambda: da.log_probs(dual(torch.zeros(4, 9)), t), lambda: da.embedding(t, dual(torch.zeros(7, 8)))):
            with pytest.raises(Exception, match="jvp|forward"):
                f()


# ---------------------------------------------------------------- references

@pytest.mark.parametrize("kind", list(decoder.ACTIVATIONS))
def test_gated_reference_agrees_with_differences(kind):
    """Central differences with h = 1e-5: curvature and rounding leave about 1e-9 of the values; 1e-7 is allowed."""
    g = torch.Generator().manual_seed(3)
    x, wg, wu, dh = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((5, 6), (7, 6), (7, 6), (5, 7)))
    r = R.gated(x, wg, wu, dh, kind)
    for t, name in ((x, "dx"), (wg, "dwg"), (wu, "dwu")):
        d, keep, f = torch.randn(t.shape, generator=g, dtype=torch.float64), t.clone(), []
        for s in (1e-5, -1e-5):
            t.copy_(keep + s * d)
            f.append((R.gated(x, wg, wu, dh, kind)["h"] * dh).sum())
        t.copy_(keep)
        assert abs((f[0] - f[1]) / 2e-5 - (r[name] * d).sum()) < 1e-7 * (1 + r[name].abs().sum())


def test_other_references_agree_with_differences():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(4, 9, generator=g, dtype=torch.float64) * 2
    x[1, 3], x[2, 5] = -math.inf, -math.inf
    t = torch.tensor([2, 4, -1, 8])
    a, b = (torch.randn(4, generator=g, dtype=torch.float64) for _ in range(2))
    r = R.log_probs(x, t, 0.7, 0, a, b)
    d, keep, f = torch.randn(x.shape, generator=g, dtype=torch.float64), x.clone(), []
    for s in (1e-5, -1e-5):
        q = R.log_probs(keep + s * d, t, 0.7)
        f.append((a * q["lp"]).sum() + (b * q["H"]).sum())
    assert abs((f[0] - f[1]) / 2e-5 - (r["dx"] * d).sum()) < 1e-7 * (1 + r["dx"].abs().sum())
    w, dy = torch.randn(6, 5, generator=g, dtype=torch.float64), torch.randn(2, 4, 5, generator=g, dtype=torch.float64)
    ids = torch.tensor([[0, 3, 3, 9], [5, 1, 3, -2]])
    r = R.embedding(ids, w, dy, 1.5, padding_idx=1)
    d = torch.randn(w.shape, generator=g, dtype=torch.float64)
    d[1] = 0
    moved = ((R.embedding(ids, w + d, dy, 1.5)["y"] - r["y"]) * dy).sum()
    assert abs(moved - (r["dw"] * d).sum()) < 1e-10 and (r["dw"][1] == 0).all()


def test_references_reject_planted_mistakes():
    """A mistake planted in a reference moves it by more than the GPU tests' tolerances."""
    g = torch.Generator().manual_seed(5)
    x, wg, wu, dh = (torch.randn(*s, generator=g).to(B16) for s in ((40, 64), (48, 64), (48, 64), (40, 48)))
    wg, wu = wg / 8, wu / 8
    r = R.gated(x, wg, wu, dh, "silu")
    tol = R.gated_tolerance(r, B16, "silu")
    late = dh.clone()
    late[-1] = 0                                                        # the last token left out
    for wrong in (R.gated(x, wg, wu, dh, "gelu"), R.gated(x, wu, wg, dh, "silu")):
        assert all(((wrong[k] - r[k]).abs() > tol[k]).any() for k in tol)
    wrong = R.gated(x, wg, wu, late, "silu")
    assert all(((wrong[k] - r[k]).abs() > tol[k]).any() for k in ("dx", "dwg", "dwu"))
    z = torch.randn(6, 300, generator=g) * 3
    t, a, b = torch.arange(6), torch.randn(6, generator=g), torch.randn(6, generator=g)
    r = R.log_probs(z, t, 1.0, 5, a, b)
    tol = R.log_probs_tolerance(r, torch.float32, 1.0)
    cut = z.clone()
    cut[:, 299] = -math.inf                                             # the last column left out
    for wrong in (R.log_probs(z, t, 1.01, 5, a, b), R.log_probs(cut, t, 1.0, 5, a, b), R.log_probs(z, (t + 1), 1.0, 5, a, -b)):
        assert ((wrong["dx"] - r["dx"]).abs() > tol["dx"]).any()
    assert all(((R.log_probs(cut, t)[k] - r[k]).abs() > tol[k]).any() for k in ("lp", "H"))
    ids, w = torch.randint(0, 9, (200,), generator=g), torch.randn(9, 4, generator=g)
    dy = torch.randn(200, 4, generator=g)
    r = R.embedding(ids, w, dy, 2.0)
    tol = R.embedding_tolerance(r, torch.float32, 2.0)
    dy[7] = 0
    assert ((R.embedding(ids, w, dy, 2.0)["dw"] - r["dw"]).abs() > tol["dw"]).any()
