"""What the binding of the training operators does around the library's calls, with a stub in the library's place: the device and
stream that a call goes to, what it takes as a workspace, what autograd is told."""
import contextlib
import ctypes
import math
import os
import sys

import pytest
import torch

import bitwise_deterministic_shard_gb300 as da
from bitwise_deterministic_shard_gb300 import train

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_train_cpu as T  # noqa: E402


class _Stub:
    """Answers every call with 0 (no workspace, no error) and notes it beside the device that was current."""

    def __init__(self):
        self.calls, self.current = [], 0

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.current, args))
            return 0
        return call


@pytest.fixture
def stub(monkeypatch):
    """CPU tensors as those of device -1 (what their get_device says), device 0 current."""
    s = _Stub()

    @contextlib.contextmanager
    def device(index):
        before, s.current = s.current, index
        yield
        s.current = before
    monkeypatch.setattr(da, "_cuda", lambda t, name: None)
    monkeypatch.setattr(da, "lib", lambda: s)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: s.current, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    return s


def _qkv():
    return [torch.zeros(1, h, 8, 64, dtype=torch.bfloat16) for h in (4, 2, 2)]


def test_calls_go_to_the_tensors_device(stub):
    """A raw stream means nothing without its device (0 is the default stream of whichever is current)."""
    q, k, v = _qkv()
    x, s = torch.zeros(4, 10), torch.zeros(4)
    da.attention_forward(q, k, v)
    da.attention_backward(q, k, v, q, torch.zeros(1, 4, 8), q)
    da.layer_norm_forward(x)
    da.layer_norm_backward(x, x, None, s, s)
    da.adamw_step([s], [s], torch.zeros(256), torch.zeros(256), 1)
    p = torch.zeros(5)
    p.grad = torch.zeros(5)
    da.AdamW([p]).step()
    launches = [c for c in stub.calls if not c[0].endswith("_bytes")]
    assert [c[0] for c in launches] == ["dta_forward", "dta_backward", "dln_forward", "dln_backward", "dow_adamw", "dow_adamw"]
    for name, device, args in launches:
        assert device == -1 and args[-1] == 1000 - 1, name
    assert stub.current == 0


# ---------------------------------------------------------------- layer norm

def test_layer_norm_weight_dtype(stub):
    x, s, w = torch.zeros(4, 10, dtype=torch.bfloat16), torch.zeros(4), torch.zeros(10)
    for weight, want, got in ((None, None, torch.bfloat16), (None, torch.float32, torch.float32), (None, x.dtype, x.dtype),
                              (w, None, torch.float32), (w, torch.float32, torch.float32), (w.bfloat16(), None, x.dtype)):
        _, dw, db = da.layer_norm_backward(x, x, weight, s, s, weight_dtype=want)
        assert dw.dtype == db.dtype == got and stub.calls[-1][2][3] == train._CODES[got]
    for weight, want in ((w, x.dtype), (w.bfloat16(), torch.float32), (None, torch.float16), (None, torch.float64)):
        with pytest.raises(da.DetAttnError):
            da.layer_norm_backward(x, x, weight, s, s, weight_dtype=want)


# ---------------------------------------------------------------- autograd

def test_forward_mode_is_refused_not_dropped(stub):
    """A dual tensor does not require a gradient; its tangent may not get lost on the way past the autograd functions."""
    q, k, v = _qkv()
    x, w, b = torch.zeros(4, 10), torch.ones(10), torch.zeros(10)
    with torch.autograd.forward_ad.dual_level():
        def dual(t):
            return torch.autograd.forward_ad.make_dual(t, torch.ones_like(t))
        for grad in (True, False):
            with torch.set_grad_enabled(grad):
                for i in range(3):
                    args = [q, k, v]
                    args[i] = dual(args[i])
                    with pytest.raises(Exception, match="jvp|forward"):
                        da.attention(*args)
                    args = [x, w, b]
                    args[i] = dual(args[i])
                    with pytest.raises(Exception, match="jvp|forward"):
                        da.layer_norm(*args)
                assert da.attention(q, k, v).shape == q.shape and da.layer_norm(x, w, b).shape == x.shape


def test_masks_and_slopes_may_not_change_before_the_backward_pass(stub):
    S, opts = 8, dict(docs=lambda: torch.zeros(1, 8, dtype=torch.int32), prefix=lambda: torch.zeros(1, dtype=torch.int32),
                      slopes=lambda: torch.zeros(4))
    for name, make in opts.items():
        q, k, v = (t.requires_grad_(True) for t in _qkv())
        t = make()
        out = da.attention(q, k, v, causal=True, **{name: t})
        out.sum().backward(retain_graph=True)
        assert q.grad.shape == q.shape and stub.calls[-1][0] == "dta_backward"
        t.add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.sum().backward()


def test_writes_through_addresses_are_seen(stub):
    """What the library writes in place counts as an in-place change: a graph that saved it refuses to go backward."""
    p, late = torch.ones(300, requires_grad=True), torch.ones(5, requires_grad=True)
    m, v, scale = torch.zeros(768), torch.zeros(768), torch.ones(1)
    y = (p * p).sum() + (late * late).sum()
    before = [t._version for t in (p, late, m, v, scale)]
    with torch.no_grad():
        da.adamw_step([p, late], [torch.ones(300), None], m, v, 1, grad_scale=scale)
    assert [t._version - b for t, b in zip((p, late, m, v, scale), before)] == [1, 0, 1, 1, 0]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    m8, s = torch.zeros(768).to(torch.float8_e4m3fn), [torch.zeros(3) for _ in range(2)]
    v8 = m8.clone()
    da.adamw_step([p.detach(), late.detach()], [torch.ones(300), torch.ones(5)], m8, v8, 1, exp_avg_scale=s[0], exp_avg_sq_scale=s[1])
    assert all(t._version for t in (m8, v8, *s))
    q, k, v = _qkv()
    out = torch.empty_like(q)
    da.attention_forward(q, k, v, out=out)
    assert out._version == 1


# ---------------------------------------------------------------- caps

@pytest.mark.parametrize("softcap, scale, code", [(0.0, 2.0 ** 100, 5), (2.0 ** -60, math.nan, 5), (2.0 ** 60, -2.0 ** 60, 5), (2.0 ** -61, math.nan, 1),
                                                  (2.0 ** 61, math.nan, 1), (-30.0, math.nan, 1), (30.0, 2.0 ** 61, 1), (1e-40, math.nan, 1)])
def test_caps_beyond_the_factors_range_are_refused(softcap, scale, code):
    """5: the arguments passed, and the workspace, which is missing, is asked for."""
    from bitwise_deterministic_shard_gb300 import build
    build.build()
    L, d, o = da.lib(), T._desc(Skv=4096, Sq=1), T._desc(Skv=4096, Sq=1)
    d.softcap, d.scale = softcap, scale
    assert L.dta_forward(ctypes.byref(d), ctypes.byref(o.q), None, None, 0, None) == code


# ---------------------------------------------------------------- AdamW

def test_adamw_counts_each_parameters_steps(stub):
    """Parameters with as many steps behind them share a launch; none without a gradient counts."""
    ps = [torch.zeros(n) for n in (5, 300, 7)]
    opt = da.AdamW(ps)
    launches = []
    for have in ((0,), (0, 1), (1,), (0, 1, 2), ()):
        for i, p in enumerate(ps):
            p.grad = torch.ones_like(p) if i in have else None
        before = len(stub.calls)
        opt.step()
        launches.append([(args[1], train._HYPER.unpack(args[9])[-1]) for _, _, args in stub.calls[before:]])
    assert launches == [[(1, 1)], [(1, 2), (1, 1)], [(1, 2)], [(2, 3), (1, 1)], []]
    assert opt.missed == [[2, 2, 4]] and opt.steps == 5


def test_adamw_refuses_a_parameter_given_twice(stub):
    p = torch.zeros(5)
    with pytest.raises(da.DetAttnError):
        da.AdamW([p, torch.zeros(5), p])


# ---------------------------------------------------------------- workspaces

def test_workspaces_are_checked(stub, monkeypatch):
    """A given workspace goes to the kernels as an address: it has to lie on the tensors' device and in one piece."""
    q, k, v = _qkv()
    s, x, lse = torch.zeros(4), torch.zeros(4, 10), torch.zeros(1, 4, 8)
    for name in ("dta_workspace_bytes", "dln_workspace_bytes"):
        setattr(stub, name, lambda *args: 4096)
    good, small = torch.zeros(4096, dtype=torch.uint8), torch.zeros(100)
    pieces = (torch.zeros(4, 8192, dtype=torch.uint8)[:, ::2], torch.zeros(1).expand(9000))
    calls = [lambda w: da.attention_forward(q, k, v, workspace=w), lambda w: da.attention_backward(q, k, v, q, lse, q, workspace=w),
             lambda w: da.layer_norm_backward(x, x, None, s, s, workspace=w)]
    for call in calls:
        for w in (good, None, small):                               # one that is too small is replaced, as elsewhere in the package
            call(w)
        assert len(stub.calls) == 3
        stub.calls.clear()
        for w in pieces:
            with pytest.raises(da.DetAttnError):
                call(w)
    elsewhere = torch.zeros(4096, dtype=torch.uint8, device="meta")

    def cuda(t, name):
        if t is elsewhere:
            raise da.DetAttnError(f"{name} must be a CUDA tensor")
    monkeypatch.setattr(da, "_cuda", cuda)
    for call in calls:
        with pytest.raises(da.DetAttnError, match="workspace"):
            call(elsewhere)
    assert not stub.calls
