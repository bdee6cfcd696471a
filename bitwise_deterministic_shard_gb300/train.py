"""Training operators of libdetattn: attention with capped, distance-biased and masked scores,
layer norm, and AdamW over many tensors, each with its gradient where it has one.

Argument marshalling only, as in the package's __init__: the computation runs in the CUDA kernels
behind include/detattn.h on the current stream, and there is no CPU path.  Every kernel adds in
an order that depends on the sizes and types alone, so equal calls give equal bytes on every run.
"""
from __future__ import annotations

import ctypes as C
import math

import torch

import bitwise_deterministic_shard_gb300 as _da
from bitwise_deterministic_shard_gb300 import DetAttnError, _Matrix, _Tensor

STATE_BLOCK = 256     # elements of an 8-bit optimizer state under one scale; tensors' states start on multiples

_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class _Train(C.Structure):
    _fields_ = [("q", _Tensor), ("k", _Tensor), ("v", _Tensor), ("causal", C.c_int32), ("scale", C.c_float),
                ("softcap", C.c_float), ("slopes", C.c_void_p), ("docs", C.c_void_p), ("prefix", C.c_void_p),
                ("dev_status", C.c_void_p)]


class _Param(C.Structure):
    _fields_ = [("param", C.c_void_p), ("grad", C.c_void_p), ("numel", C.c_int64), ("state", C.c_int64)]


class _Hyper(C.Structure):
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double), ("eps", C.c_double),
                ("weight_decay", C.c_double), ("step", C.c_int64)]


_NAMES = ("dta_forward", "dta_backward", "dln_forward", "dln_backward", "dow_adamw")


def declare(L):
    """Argument types of the training entry points of a loaded library."""
    P, T, M, I = C.c_void_p, C.POINTER(_Tensor), C.POINTER(_Matrix), C.c_int
    D = C.POINTER(_Train)
    L.dta_workspace_bytes.argtypes, L.dta_workspace_bytes.restype = [D, I], C.c_size_t
    L.dta_forward.argtypes = [D, T, P, P, C.c_size_t, P]
    L.dta_backward.argtypes = [D, T, P, T, T, T, T, P, C.c_size_t, P]
    L.dln_forward.argtypes = [M, P, P, I, C.c_float, M, P, P, P]
    L.dln_workspace_bytes.argtypes, L.dln_workspace_bytes.restype = [C.c_int64, C.c_int64], C.c_size_t
    L.dln_backward.argtypes = [M, M, P, I, P, P, M, P, P, P, C.c_size_t, P]
    L.dow_adamw.argtypes = [C.POINTER(_Param), I, I, I, P, P, P, P, C.c_int64, C.POINTER(_Hyper), P, P]
    for f in _NAMES:
        getattr(L, f).restype = C.c_int


def _code(t, name, allowed=_CODES):
    c = allowed.get(t.dtype)
    if c is None:
        raise DetAttnError(f"{name}: unsupported dtype {t.dtype}")
    return c


def _same_device(device, **ts):
    for name, t in ts.items():
        if t is not None:
            _da._cuda(t, name)
            if t.device != device:
                raise DetAttnError(f"{name} is on {t.device}, expected {device}")


# ---------------------------------------------------------------- attention

_HALF = {torch.bfloat16: 1, torch.float16: 2}


def _ready(t):
    """t in a layout that the kernels' tensor maps can describe: itself, or a contiguous copy (a
    last dimension that is not contiguous, broadcast dimensions, strides or starts off 16 bytes)."""
    st, sh = t.stride(), t.shape
    if (st[3] == 1 and t.data_ptr() % 16 == 0
            and all(n <= 1 or (x > 0 and x % 8 == 0) for n, x in zip(sh[:3], st[:3]))):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _view4(t, name, code) -> _Tensor:
    x = _Tensor()
    x.ptr, x.dtype = t.data_ptr(), code
    x.B, x.H, x.S, x.D = t.shape
    x.stride[:] = t.stride()
    return x


class _Attention:
    """Checked arguments of one attention call; keeps the tensors alive while it lives."""

    def __init__(self, Q, K, V, causal, scale, softcap, slopes, docs, prefix, status):
        for t, name in ((Q, "Q"), (K, "K"), (V, "V")):
            _da._cuda(t, name)
            if t.dim() != 4:
                raise DetAttnError(f"{name} must be [B, H, S, D]")
        code = _code(Q, "Q", _HALF)
        if K.dtype != Q.dtype or V.dtype != Q.dtype:
            raise DetAttnError("Q, K and V must share one dtype (bf16 or f16)")
        self.device, dev = Q.device, Q.device
        _same_device(dev, K=K, V=V, slopes=slopes, docs=docs, prefix=prefix, status=status)
        self.B, self.Hq, self.Sq, self.D = Q.shape
        _, self.Hkv, self.Skv, _ = K.shape
        if slopes is not None and (slopes.dtype != torch.float32 or tuple(slopes.shape) != (self.Hq,)):
            raise DetAttnError(f"slopes must be f32 [{self.Hq}]")
        if slopes is not None and slopes.requires_grad:
            raise DetAttnError("slopes have no gradient: pass them detached")
        if docs is not None and (docs.dtype != torch.int32 or tuple(docs.shape) != (self.B, self.Skv)):
            raise DetAttnError(f"docs must be int32 [{self.B}, {self.Skv}]")
        if prefix is not None and (prefix.dtype != torch.int32 or tuple(prefix.shape) != (self.B,)):
            raise DetAttnError(f"prefix must be int32 [{self.B}]")
        slopes, docs, prefix = (None if t is None else t.contiguous() for t in (slopes, docs, prefix))
        q, k, v = (_ready(t.detach()) for t in (Q, K, V))
        self.keep = [q, k, v, slopes, docs, prefix]
        self.code = code
        d = self.desc = _Train()
        d.q, d.k, d.v = _view4(q, "Q", code), _view4(k, "K", code), _view4(v, "V", code)
        d.causal = 1 if causal else 0
        d.scale = math.nan if scale is None else float(scale)
        d.softcap = float(softcap)
        d.slopes, d.docs, d.prefix = _addr(slopes), _addr(docs), _addr(prefix)
        d.dev_status = None if status is None else _da._sptr(status).value

    def workspace(self, backward, ws):
        need = int(_da.lib().dta_workspace_bytes(C.byref(self.desc), backward))
        if ws is None or ws.numel() * ws.element_size() < need:
            ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        return ws, need


def _addr(t):
    return None if t is None else t.data_ptr()


def _like(t):
    """An uninitialised tensor of t's layout where that is dense and fit for the kernels, else contiguous."""
    o = torch.empty_like(t)
    return o if _ready_layout(o) else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _ready_layout(t):
    return t.stride(3) == 1 and all(n <= 1 or (x > 0 and x % 8 == 0) for n, x in zip(t.shape[:3], t.stride()[:3]))


def _given(out, like, name):
    if out is None:
        return _like(like)
    _da._cuda(out, name)
    if (out.dtype != like.dtype or out.shape != like.shape or out.device != like.device or not _ready_layout(out)
            or out.data_ptr() % 16):
        raise DetAttnError(f"{name} must be {like.dtype} {tuple(like.shape)} on {like.device}, 16-byte aligned, "
                           "its last dimension contiguous and its other strides multiples of 8")
    return out


def attention_forward(Q, K, V, causal=False, scale=None, softcap=0.0, slopes=None, docs=None, prefix=None, out=None,
                      workspace=None, status=None, need_lse=True):
    """Attention with capped, distance-biased and masked scores: (out [B, Hq, Sq, D], lse f32 [B, Hq, Sq]).

    Q [B, Hq, Sq, D], K and V [B, Hkv, Skv, D], all bf16 or all f16, D a multiple of 8 up to 128; query
    head h reads key head h // (Hq // Hkv); query i stands at position i + Skv - Sq.
      t = scale q.k (scale: 1/sqrt(D));  u = softcap tanh(t / softcap), softcap = 0: t
      s = u - slopes[h] |position - j|   (slopes: f32 [Hq])
    A query sees key j when not causal, or j <= its position, or j < prefix[b] (int32 [B], with causal
    only), and, with docs (int32 [B, Skv]), when both tokens have the same id >= 0.  A query that
    sees nothing gets zeros and lse = -inf.  Few queries (Sq * Hq / Hkv <= 128) read the keys once per
    key head, split over the GPU.  out takes Q's layout."""
    A = _Attention(Q, K, V, causal, scale, softcap, slopes, docs, prefix, status)
    out = _given(out, Q.detach(), "out")
    lse = torch.empty((A.B, A.Hq, A.Sq), dtype=torch.float32, device=A.device) if need_lse else None
    ws, need = A.workspace(0, workspace)
    o = _view4(out, "out", A.code)
    _da._check(_da.lib().dta_forward(C.byref(A.desc), C.byref(o), _addr(lse), _addr(ws), need, _da._stream()),
               "attention_forward")
    return out, lse


def attention_backward(Q, K, V, out, lse, grad, causal=False, scale=None, softcap=0.0, slopes=None, docs=None, prefix=None,
                       workspace=None, status=None):
    """(dQ, dK, dV) of sum(out * grad) from attention_forward's out and lse; the other arguments as there.
    The gradient of a shared key head is the sum over its query heads, formed in binary32."""
    A = _Attention(Q, K, V, causal, scale, softcap, slopes, docs, prefix, status)
    for t, name in ((out, "out"), (grad, "grad")):
        _da._cuda(t, name)
        if t.dtype != Q.dtype or t.shape != Q.shape or t.device != Q.device:
            raise DetAttnError(f"{name} must be {Q.dtype} {tuple(Q.shape)} on {Q.device}")
    _da._cuda(lse, "lse")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (A.B, A.Hq, A.Sq) or lse.device != A.device:
        raise DetAttnError(f"lse must be f32 {(A.B, A.Hq, A.Sq)} on {A.device}")
    out, grad, lse = _ready(out.detach()), _ready(grad.detach()), lse.contiguous()
    dq, dk, dv = (_like(t.detach()) for t in (Q, K, V))
    ws, need = A.workspace(1, workspace)
    v = [_view4(t, "", A.code) for t in (out, grad, dq, dk, dv)]
    _da._check(_da.lib().dta_backward(C.byref(A.desc), C.byref(v[0]), _addr(lse), C.byref(v[1]), C.byref(v[2]), C.byref(v[3]),
                                      C.byref(v[4]), _addr(ws), need, _da._stream()), "attention_backward")
    return dq, dk, dv


class _AttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, V, kw):
        out, lse = attention_forward(Q, K, V, **kw)
        ctx.save_for_backward(Q, K, V, out, lse)
        ctx.kw = kw
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        return (*attention_backward(*ctx.saved_tensors, grad, **ctx.kw), None)


def attention(Q, K, V, causal=False, scale=None, softcap=0.0, slopes=None, docs=None, prefix=None, status=None):
    """attention_forward's output, with autograd for Q, K and V.  (A backward pass that is captured into a
    CUDA graph calls attention_backward itself, as with any autograd function whose leaves live in
    an eager graph too.)"""
    kw = dict(causal=causal, scale=scale, softcap=softcap, slopes=slopes, docs=docs, prefix=prefix, status=status)
    if torch.is_grad_enabled() and (Q.requires_grad or K.requires_grad or V.requires_grad):
        return _AttentionFn.apply(Q, K, V, kw)
    return attention_forward(Q, K, V, need_lse=False, **kw)[0]


# ---------------------------------------------------------------- layer norm

def _rows(t, name, code):
    """t [..., cols] as a matrix of rows: itself where one row stride describes it, else a contiguous copy."""
    cols = t.shape[-1]
    if t.is_contiguous():
        n = t.numel() // cols if cols else 0
        stride = cols
    else:
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < cols):
            t = t.contiguous() if t.dim() == 1 or t.stride(-1) != 1 or not _even(t) else t
        n = t.numel() // cols if cols else 0
        stride = t.stride(-2) if t.dim() > 1 and n > 1 and t.shape[-2] > 1 else cols
        if t.is_contiguous():
            stride = cols
    m = _Matrix()
    m.ptr, m.dtype, m.rows, m.cols, m.row_stride = t.data_ptr(), code, n, cols, stride
    return m, t


def _even(t):
    """Whether the leading dimensions of t are one run of rows at the stride of its last but one."""
    want = t.stride(-2)
    if want < t.shape[-1]:
        return False
    for i in range(t.dim() - 2, -1, -1):
        if t.shape[i] > 1 and t.stride(i) != want:
            return False
        want *= t.shape[i]
    return True


def _weights(x, weight, bias):
    cols = x.shape[-1] if x.dim() else 0
    if cols < 1:
        raise DetAttnError("x must be [..., cols] with at least one column")
    code = _code(x, "x")
    wt = None
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        if tuple(t.shape) != (cols,) or t.dtype not in (x.dtype, torch.float32):
            raise DetAttnError(f"{name} must be [{cols}] of x's dtype or f32")
        if wt is not None and t.dtype != wt:
            raise DetAttnError("weight and bias must share one dtype")
        wt = t.dtype
    _same_device(x.device, weight=weight, bias=bias)
    return cols, code, wt or x.dtype


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5):
    """Layer norm over the last dimension: (y like x, mean f32, rstd f32, one per row).
    x [..., cols] f32, bf16 or f16; weight and bias [cols] of x's dtype or f32, or None."""
    _da._cuda(x, "x")
    cols, code, wt = _weights(x, weight, bias)
    X, x = _rows(x.detach(), "x", code)
    weight, bias = (None if t is None else t.detach().contiguous() for t in (weight, bias))
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    Y, _ = _rows(y, "y", code)
    mean, rstd = torch.empty((2, *x.shape[:-1]), dtype=torch.float32, device=x.device).unbind(0)
    _da._check(_da.lib().dln_forward(C.byref(X), _addr(weight), _addr(bias), _CODES[wt], eps, C.byref(Y), _addr(mean),
                                     _addr(rstd), _da._stream()), "layer_norm_forward")
    return y, mean, rstd


def layer_norm_backward(grad, x, weight, mean, rstd, need_weight=True, need_bias=True, workspace=None):
    """(dx, dweight, dbias) from the upstream gradient and layer_norm_forward's mean and rstd; the
    weight gradients are None where not needed, and of weight's dtype (x's without a weight)."""
    _da._cuda(grad, "grad")
    _da._cuda(x, "x")
    cols, code, wt = _weights(x, weight, None)
    if grad.shape != x.shape or grad.dtype != x.dtype:
        raise DetAttnError("grad must have x's shape and dtype")
    rows = x.numel() // cols
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _da._cuda(t, name)
        if t.dtype != torch.float32 or t.numel() != rows or not t.is_contiguous():
            raise DetAttnError(f"{name} must be contiguous f32 with one entry per row")
    _same_device(x.device, grad=grad, mean=mean, rstd=rstd)
    X, x = _rows(x.detach(), "x", code)
    G, grad = _rows(grad.detach(), "grad", code)
    weight = None if weight is None else weight.detach().contiguous()
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    DX, _ = _rows(dx, "dx", code)
    dw = torch.empty(cols, dtype=wt, device=x.device) if need_weight else None
    db = torch.empty(cols, dtype=wt, device=x.device) if need_bias else None
    L = _da.lib()
    need = int(L.dln_workspace_bytes(rows, cols)) if need_weight or need_bias else 0
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _da._check(L.dln_backward(C.byref(G), C.byref(X), _addr(weight), _CODES[wt], _addr(mean), _addr(rstd), C.byref(DX),
                              _addr(dw), _addr(db), _addr(workspace) if need else None, need, _da._stream()),
               "layer_norm_backward")
    return dx, dw, db


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = layer_norm_backward(grad, x, weight, mean, rstd, need[1], need[2])
        if db is not None and db.dtype != ctx.bias_dtype:
            db = db.to(ctx.bias_dtype)
        return dx if need[0] else None, dw, db, None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """layer_norm_forward's y, with autograd for x, weight and bias."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (x, weight, bias)):
        return _LayerNorm.apply(x, weight, bias, eps)
    return layer_norm_forward(x, weight, bias, eps)[0]


# ---------------------------------------------------------------- AdamW

def adamw_state_len(params) -> int:
    """Elements of the state arrays of adamw_step: each tensor's start on a multiple of STATE_BLOCK."""
    return sum(-(-p.numel() // STATE_BLOCK) * STATE_BLOCK for p in params)


def adamw_step(params, grads, exp_avg, exp_avg_sq, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2,
               exp_avg_scale=None, exp_avg_sq_scale=None, grad_scale=None):
    """One AdamW step over many tensors, in place, in one launch for up to 120 of them.

    params, grads: contiguous tensors of one dtype (f32, bf16, f16); a grad of None leaves its tensor as it is.
    exp_avg, exp_avg_sq: [adamw_state_len(params)], tensor after tensor, each from the next multiple of
    STATE_BLOCK on: f32, or float8_e4m3fn with f32 scales [len / STATE_BLOCK] in exp_avg_scale and
    exp_avg_sq_scale (exp_avg_sq then holds the square root; zeros, scales included, are the initial state).
    step: 1 on the first call.  grad_scale: optional f32 CUDA scalar that multiplies every gradient.
    Every operation is rounded once to binary32; the hyperparameters are baked into the launch, so a
    captured graph replays this step's."""
    params, grads = list(params), list(grads)
    if len(params) != len(grads):
        raise DetAttnError("params and grads must have the same length")
    if not params:
        return
    dt, dev = params[0].dtype, params[0].device
    code = _code(params[0], "params")
    n = len(params)
    table = (_Param * n)()
    at = k = 0
    for p, g in zip(params, grads):
        if p.dtype != dt or p.device != dev or not p.is_contiguous():
            raise DetAttnError("params must be contiguous tensors of one dtype on one device")
        m = p.numel()
        if g is not None:
            if g.dtype != dt or g.device != dev or g.numel() != m or not g.is_contiguous():
                raise DetAttnError("grads must be contiguous, of their params' dtype, device and size")
            e = table[k]
            e.param, e.grad, e.numel, e.state = p.data_ptr(), g.data_ptr(), m, at
            k += 1
        at += -(-m // STATE_BLOCK) * STATE_BLOCK
    _da._cuda(params[0], "params")
    bits = 8 if exp_avg.dtype == torch.float8_e4m3fn else 32
    st = torch.float8_e4m3fn if bits == 8 else torch.float32
    for t, name, want, length in ((exp_avg, "exp_avg", st, at), (exp_avg_sq, "exp_avg_sq", st, at),
                                  (exp_avg_scale, "exp_avg_scale", torch.float32, at // STATE_BLOCK),
                                  (exp_avg_sq_scale, "exp_avg_sq_scale", torch.float32, at // STATE_BLOCK)):
        if name.endswith("scale") and bits == 32:
            if t is not None:
                raise DetAttnError("scales go with 8-bit states")
            continue
        if t is None or t.dtype != want or t.numel() != length or not t.is_contiguous() or t.device != dev:
            raise DetAttnError(f"{name} must be contiguous {want} [{length}] on {dev}")
    if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1 or grad_scale.device != dev):
        raise DetAttnError(f"grad_scale must be one f32 element on {dev}")
    h = _Hyper(lr, betas[0], betas[1], eps, weight_decay, int(step))
    _da._check(_da.lib().dow_adamw(table, k, code, bits, _addr(exp_avg), _addr(exp_avg_sq), _addr(exp_avg_scale),
                                   _addr(exp_avg_sq_scale), at, C.byref(h), _addr(grad_scale), _da._stream()), "adamw_step")


class AdamW:
    """AdamW over a list of parameters, grouped by dtype, with f32 or 8-bit states (adamw_step)."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=32):
        if state_bits not in (8, 32):
            raise DetAttnError("state_bits must be 8 or 32")
        self.hyper = dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay)
        self.state_bits, self.steps, self.groups = state_bits, 0, []
        by = {}
        for p in params:
            by.setdefault((p.dtype, p.device), []).append(p)
        for (_, dev), ps in by.items():
            n = adamw_state_len(ps)
            kw = dict(dtype=torch.float8_e4m3fn if state_bits == 8 else torch.float32, device=dev)
            g = {"params": ps, "exp_avg": torch.zeros(n, **kw), "exp_avg_sq": torch.zeros(n, **kw)}
            if state_bits == 8:
                g["exp_avg_scale"], g["exp_avg_sq_scale"] = torch.zeros((2, n // STATE_BLOCK), device=dev).unbind(0)
            self.groups.append(g)

    def step(self, grad_scale=None):
        self.steps += 1
        for g in self.groups:
            ps = g["params"]
            with torch.no_grad():
                adamw_step(ps, [None if p.grad is None else p.grad.contiguous() for p in ps], g["exp_avg"], g["exp_avg_sq"],
                           self.steps, exp_avg_scale=g.get("exp_avg_scale"), exp_avg_sq_scale=g.get("exp_avg_sq_scale"),
                           grad_scale=grad_scale, **self.hyper)

    def zero_grad(self):
        for g in self.groups:
            for p in g["params"]:
                p.grad = None
