"""Training operators of libdetattn: attention with capped, distance-biased and masked scores,
layer norm, and AdamW over many tensors, each with its gradient where it has one.

Argument marshalling only, as in the package's __init__: the computation runs in the CUDA kernels
behind include/detattn.h on the current stream of the tensors' device, and there is no CPU path.  Every kernel adds in
an order that depends on the sizes, types and options and, for layer norm, on what starts on 16 bytes, so equal calls (for
layer norm: on equally aligned tensors) give equal bytes on every run.
"""
from __future__ import annotations

import ctypes as C
import math
import struct

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


# The same structures as bytes: one pack is several times cheaper than filling a ctypes structure, and
# the smallest calls here take no longer on the GPU than their arguments on the host.
_TENSOR, _DESC, _MATRIX, _HYPER = (struct.Struct(f) for f in ("Pi8q", "Pi8q" * 3 + "iffPPPP", "Pi3q", "5dq"))


_NAMES = ("dta_forward", "dta_backward", "dln_forward", "dln_backward", "dow_adamw")


def declare(L):
    """Argument types of the training entry points of a loaded library."""
    P, I, N = C.c_void_p, C.c_int, C.c_size_t
    L.dta_workspace_bytes.argtypes, L.dta_workspace_bytes.restype = [P, I], N
    L.dta_forward.argtypes = [P, P, P, P, N, P]
    L.dta_backward.argtypes = [P, P, P, P, P, P, P, P, N, P]
    L.dln_forward.argtypes = [P, P, P, I, C.c_float, P, P, P, P]
    L.dln_workspace_bytes.argtypes, L.dln_workspace_bytes.restype = [C.c_int64, C.c_int64], N
    L.dln_backward.argtypes = [P, P, P, I, P, P, P, P, P, P, N, P]
    L.dow_adamw.argtypes = [P, I, I, I, P, P, P, P, C.c_int64, P, P, P]
    for f in _NAMES:
        getattr(L, f).restype = C.c_int


def _code(t, name, allowed=_CODES):
    c = allowed.get(t.dtype)
    if c is None:
        raise DetAttnError(f"{name}: unsupported dtype {t.dtype}")
    return c


def _on(index, name, t):
    """t on the device of that index (as torch.Tensor.get_device gives it)."""
    _da._cuda(t, name)
    if t.get_device() != index:
        raise DetAttnError(f"{name} is on another device")


def _run(what, index, f, *args):
    """f(*args, stream) on the current stream of the tensors' device, with that device current: a launch goes to the
    current one, whichever device its addresses and its stream belong to."""
    if torch._C._cuda_getDevice() == index:
        code = f(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            code = f(*args, torch._C._cuda_getCurrentRawStream(index))
    _da._check(code, what)


def _tracked(*ts):
    """Whether autograd may follow any of ts: backward, or forward mode, whose tensors do not require a gradient (its
    functions then refuse, as they have no forward-mode derivative)."""
    if torch.autograd.forward_ad._current_level >= 0:
        return True
    for t in ts:
        if t is not None and t.requires_grad:
            return torch.is_grad_enabled()
    return False


def _written(ts):
    """Tells autograd of writes that went through addresses: a graph that saved one of ts refuses to go backward."""
    torch.autograd.graph.increment_version(ts)


def _addr(t):
    return None if t is None else t.data_ptr()


def _room(need, ws, device, index):
    """ws where it holds need bytes, else a new workspace."""
    if ws is None or ws.numel() * ws.element_size() < need:
        return torch.empty(need, dtype=torch.uint8, device=device) if need else None
    _on(index, "workspace", ws)
    if not ws.is_contiguous():
        raise DetAttnError("workspace must be contiguous")
    return ws


# ---------------------------------------------------------------- attention

_HALF = {torch.bfloat16: 1, torch.float16: 2}


def _fits(t):
    """Whether the kernels' tensor maps can describe t: its last dimension contiguous, its start on 16 bytes, its
    other strides multiples of 8 and not zero (where the dimension is longer than 1)."""
    s0, s1, s2, s3 = t.stride()
    if t.data_ptr() & 15 or s3 != 1:
        return False
    if s0 > 0 and s1 > 0 and s2 > 0 and not (s0 | s1 | s2) & 7:
        return True
    return all(n <= 1 or (x > 0 and x % 8 == 0) for n, x in zip(t.shape, (s0, s1, s2)))


def _ready(t):
    """t itself where it fits, else a contiguous copy."""
    return t if _fits(t) else t.detach().clone(memory_format=torch.contiguous_format)


def _view(t, code):
    return _TENSOR.pack(t.data_ptr(), code, *t.shape, *t.stride())


def _option(t, name, dtype, shape, index):
    _on(index, name, t)
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise DetAttnError(f"{name} must be {dtype} {list(shape)}")
    return t if t.is_contiguous() else t.contiguous()


class _Attention:
    """Checked arguments of one attention call; keeps the tensors alive while it lives."""
    __slots__ = ("desc", "keep", "code", "index", "device", "shape")

    def __init__(self, Q, K, V, causal, scale, softcap, slopes, docs, prefix, status):
        _da._cuda(Q, "Q")
        index = self.index = Q.get_device()
        if K.get_device() != index or V.get_device() != index:
            raise DetAttnError("Q, K and V must be CUDA tensors on one device")
        dt, shape, kshape = Q.dtype, Q.shape, K.shape
        if len(shape) != 4 or len(kshape) != 4 or V.dim() != 4:
            raise DetAttnError("Q, K and V must be [B, H, S, D]")
        code = self.code = _HALF.get(dt, 0)
        if not code or K.dtype != dt or V.dtype != dt:
            raise DetAttnError(f"Q, K and V must share one dtype (bf16 or f16), not {dt}, {K.dtype}, {V.dtype}")
        self.device, self.shape = Q.device, shape
        slopes_at = docs_at = prefix_at = status_at = 0
        if slopes is not None:
            if slopes.requires_grad:
                raise DetAttnError("slopes have no gradient: pass them detached")
            slopes = _option(slopes, "slopes", torch.float32, (shape[1],), index)
            slopes_at = slopes.data_ptr()
        if docs is not None:
            docs = _option(docs, "docs", torch.int32, (shape[0], kshape[2]), index)
            docs_at = docs.data_ptr()
        if prefix is not None:
            prefix = _option(prefix, "prefix", torch.int32, (shape[0],), index)
            prefix_at = prefix.data_ptr()
        if status is not None:
            _on(index, "status", status)
            status_at = _da._sptr(status).value
        q, k, v = _ready(Q), _ready(K), _ready(V)
        self.keep = (q, k, v, slopes, docs, prefix)
        self.desc = _DESC.pack(q.data_ptr(), code, *shape, *q.stride(), k.data_ptr(), code, *kshape, *k.stride(),
                               v.data_ptr(), code, *v.shape, *v.stride(), 1 if causal else 0,
                               math.nan if scale is None else scale, softcap, slopes_at, docs_at, prefix_at, status_at)


def _like(t):
    """An uninitialised tensor of t's layout where that is dense and fit for the kernels, else contiguous."""
    o = torch.empty_like(t)
    return o if _fits(o) else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _given(out, like, name):
    if out is None:
        return _like(like)
    _da._cuda(out, name)
    if out.dtype != like.dtype or out.shape != like.shape or out.device != like.device or not _fits(out):
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
    key head, split over the GPU.  out takes Q's layout.  Tensors that the kernels cannot address (a last
    dimension that is not contiguous, strides or starts off 16 bytes, broadcast dimensions) are copied."""
    A = _Attention(Q, K, V, causal, scale, softcap, slopes, docs, prefix, status)
    given, out = out, _given(out, Q, "out")
    lse = torch.empty(A.shape[:3], dtype=torch.float32, device=A.device) if need_lse else None
    L = _da.lib()
    need = L.dta_workspace_bytes(A.desc, 0)
    ws = _room(need, workspace, A.device, A.index)
    _run("attention_forward", A.index, L.dta_forward, A.desc, _view(out, A.code), _addr(lse), _addr(ws), need)
    if given is not None:
        _written(out)
    return out, lse


def attention_backward(Q, K, V, out, lse, grad, causal=False, scale=None, softcap=0.0, slopes=None, docs=None, prefix=None,
                       workspace=None, status=None):
    """(dQ, dK, dV) of sum(out * grad) from attention_forward's out and lse; the other arguments as there.
    The gradient of a shared key head is the sum over its query heads, formed in binary32."""
    A = _Attention(Q, K, V, causal, scale, softcap, slopes, docs, prefix, status)
    index, shape, dt = A.index, A.shape, Q.dtype
    for t in (out, grad):
        if t.get_device() != index or t.dtype != dt or t.shape != shape:
            raise DetAttnError(f"out and grad must be {dt} {tuple(shape)} on Q's device")
    if lse.get_device() != index or lse.dtype != torch.float32 or lse.shape != shape[:3]:
        raise DetAttnError(f"lse must be f32 {tuple(shape[:3])} on Q's device")
    out, grad = _ready(out), _ready(grad)
    if not lse.is_contiguous():
        lse = lse.contiguous()
    dq, dk, dv = _like(Q), _like(K), _like(V)
    L, c = _da.lib(), A.code
    need = L.dta_workspace_bytes(A.desc, 1)
    ws = _room(need, workspace, A.device, A.index)
    _run("attention_backward", index, L.dta_backward, A.desc, _view(out, c), lse.data_ptr(), _view(grad, c), _view(dq, c),
         _view(dk, c), _view(dv, c), _addr(ws), need)
    return dq, dk, dv


class _AttentionFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, V, slopes, docs, prefix, kw):
        out, lse = attention_forward(Q, K, V, slopes=slopes, docs=docs, prefix=prefix, **kw)
        ctx.save_for_backward(Q, K, V, out, lse, slopes, docs, prefix)   # a change in place of any of them is refused
        ctx.kw = kw
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        Q, K, V, out, lse, slopes, docs, prefix = ctx.saved_tensors
        return (*attention_backward(Q, K, V, out, lse, grad, slopes=slopes, docs=docs, prefix=prefix, **ctx.kw),
                None, None, None, None)


def attention(Q, K, V, causal=False, scale=None, softcap=0.0, slopes=None, docs=None, prefix=None, status=None):
    """attention_forward's output, with autograd for Q, K and V.  (A backward pass that is captured into a
    CUDA graph calls attention_backward itself, as with any autograd function whose leaves live in
    an eager graph too.)"""
    kw = dict(causal=causal, scale=scale, softcap=softcap, status=status)
    if _tracked(Q, K, V):
        return _AttentionFn.apply(Q, K, V, slopes, docs, prefix, kw)
    return attention_forward(Q, K, V, slopes=slopes, docs=docs, prefix=prefix, need_lse=False, **kw)[0]


# ---------------------------------------------------------------- layer norm

def _rows(t, code, cols):
    """t [..., cols] as the bytes of a matrix of rows, and t: itself where one row stride describes it, else a
    contiguous copy."""
    n = t.numel() // cols
    if t.is_contiguous():
        return _MATRIX.pack(t.data_ptr(), code, n, cols, cols), t
    if t.dim() > 1 and (cols == 1 or t.stride(-1) == 1):
        # the leading dimensions as one run of rows: strides of those longer than 1, from the last on
        run = want = None
        for i in range(t.dim() - 2, -1, -1):
            if t.shape[i] > 1:
                if run is None:
                    run = want = t.stride(i)
                if t.stride(i) != want:
                    run = -1
                    break
                want *= t.shape[i]
        if run is None or run >= cols:
            return _MATRIX.pack(t.data_ptr(), code, n, cols, cols if run is None else run), t
    t = t.detach().contiguous()
    return _MATRIX.pack(t.data_ptr(), code, n, cols, cols), t


def _weights(x, weight, bias):
    _da._cuda(x, "x")
    shape, dt = x.shape, x.dtype
    cols = shape[-1] if shape else 0
    if cols < 1:
        raise DetAttnError("x must be [..., cols] with at least one column")
    code, index = _code(x, "x"), x.get_device()
    wt = None
    for t in (weight, bias):
        if t is None:
            continue
        kind = t.dtype
        if t.get_device() != index or t.dim() != 1 or t.shape[0] != cols or (kind != dt and kind != torch.float32):
            raise DetAttnError(f"weight and bias must be [{cols}] of x's dtype or f32, on its device")
        if wt is not None and kind != wt:
            raise DetAttnError("weight and bias must share one dtype")
        wt = kind
    return cols, code, wt or dt, index


def _packed(t):
    return t if t is None or t.is_contiguous() else t.detach().contiguous()


def layer_norm_forward(x, weight=None, bias=None, eps=1e-5, need_stats=True):
    """Layer norm over the last dimension: (y like x, mean f32, rstd f32, one per row).
    x [..., cols] f32, bf16 or f16; weight and bias [cols] of x's dtype or f32, or None.  mean and rstd, which
    the backward pass takes, are None without need_stats.  Rows, weight and bias that all start on 16 bytes are added up in
    another order than others: the same values in a shifted view can differ in low bits."""
    cols, code, wt, index = _weights(x, weight, bias)
    X, x = _rows(x, code, cols)
    weight, bias = _packed(weight), _packed(bias)
    shape, dev = x.shape, x.device
    y = torch.empty(shape, dtype=x.dtype, device=dev)
    mean = rstd = None
    if need_stats:
        mean = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
        rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev)
    Y = _MATRIX.pack(y.data_ptr(), code, y.numel() // cols, cols, cols)
    _run("layer_norm_forward", index, _da.lib().dln_forward, X, _addr(weight), _addr(bias), _CODES[wt], eps, Y, _addr(mean),
         _addr(rstd))
    return y, mean, rstd


def layer_norm_backward(grad, x, weight, mean, rstd, need_weight=True, need_bias=True, workspace=None, weight_dtype=None):
    """(dx, dweight, dbias) from the upstream gradient and layer_norm_forward's mean and rstd; the
    weight gradients are None where not needed, and of weight's dtype; without a weight of weight_dtype, x's or f32
    (None: x's), such as the dtype of a bias that has no weight beside it."""
    cols, code, wt, index = _weights(x, weight, None)
    if weight_dtype is not None and weight_dtype != wt:
        if weight is not None or weight_dtype != torch.float32:
            raise DetAttnError("weight_dtype must be weight's dtype, without a weight x's or f32")
        wt = weight_dtype
    if grad.get_device() != index or grad.shape != x.shape or grad.dtype != x.dtype:
        raise DetAttnError("grad must have x's shape, dtype and device")
    rows = x.numel() // cols
    for t in (mean, rstd):
        if t.get_device() != index or t.dtype != torch.float32 or t.numel() != rows or not t.is_contiguous():
            raise DetAttnError("mean and rstd must be contiguous f32 with one entry per row, on x's device")
    X, x = _rows(x, code, cols)
    G, grad = _rows(grad, code, cols)
    weight = _packed(weight)
    dev = x.device
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    DX = _MATRIX.pack(dx.data_ptr(), code, rows, cols, cols)
    dw = torch.empty(cols, dtype=wt, device=dev) if need_weight else None
    db = torch.empty(cols, dtype=wt, device=dev) if need_bias else None
    L = _da.lib()
    need = L.dln_workspace_bytes(rows, cols) if need_weight or need_bias else 0
    ws = _room(need, workspace, dev, index)
    _run("layer_norm_backward", index, L.dln_backward, G, X, _addr(weight), _CODES[wt], mean.data_ptr(), rstd.data_ptr(), DX,
         _addr(dw), _addr(db), _addr(ws), need)
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
        dx, dw, db = layer_norm_backward(grad, x, weight, mean, rstd, need[1], need[2],
                                         weight_dtype=ctx.bias_dtype if need[2] else None)
        return dx if need[0] else None, dw, db, None


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """layer_norm_forward's y, with autograd for x, weight and bias."""
    if _tracked(x, weight, bias):
        return _LayerNorm.apply(x, weight, bias, eps)
    return layer_norm_forward(x, weight, bias, eps, need_stats=False)[0]


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
    exp_avg_sq_scale (exp_avg_sq then holds the square root; zeros, scales included, are the initial state;
    what is not finite becomes NaN in its own element).
    step: 1 on the first call.  grad_scale: optional f32 CUDA scalar that multiplies every gradient.
    Every operation is rounded once to binary32; the hyperparameters are baked into the launch, so a
    captured graph replays this step's."""
    params, grads = list(params), list(grads)
    if len(params) != len(grads):
        raise DetAttnError("params and grads must have the same length")
    if not params:
        return
    dt, index = params[0].dtype, params[0].get_device()
    code = _code(params[0], "params")
    _da._cuda(params[0], "params")
    table, moved, at, block = [], [], 0, STATE_BLOCK
    for p, g in zip(params, grads):
        if p.dtype is not dt or p.get_device() != index or not p.is_contiguous():
            raise DetAttnError("params must be contiguous tensors of one dtype on one device")
        m = p.numel()
        if g is not None:
            if g.dtype is not dt or g.numel() != m or g.get_device() != index or not g.is_contiguous():
                raise DetAttnError("grads must be contiguous, of their params' dtype, device and size")
            table += (p.data_ptr(), g.data_ptr(), m, at)
            moved.append(p)
        at += (m + block - 1) // block * block
    states = (exp_avg, exp_avg_sq)
    if exp_avg.dtype == torch.float8_e4m3fn:
        bits, scales = 8, (exp_avg_scale, exp_avg_sq_scale)
    else:
        bits, scales = 32, ()
        if exp_avg_scale is not None or exp_avg_sq_scale is not None:
            raise DetAttnError("scales go with 8-bit states")
    for ts, want, length in ((states, torch.float8_e4m3fn if bits == 8 else torch.float32, at), (scales, torch.float32, at // block)):
        for t in ts:
            if t is None or t.dtype != want or t.numel() != length or not t.is_contiguous() or t.get_device() != index:
                raise DetAttnError(f"exp_avg{'_scale' if ts is scales else ''} and exp_avg_sq{'_scale' if ts is scales else ''} "
                                   f"must be contiguous {want} [{length}] on the params' device")
    if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1
                                   or grad_scale.get_device() != index):
        raise DetAttnError("grad_scale must be one f32 element on the params' device")
    k = len(table) // 4
    _run("adamw_step", index, _da.lib().dow_adamw, struct.pack(f"{4 * k}Q", *table), k, code, bits, exp_avg.data_ptr(),
         exp_avg_sq.data_ptr(), _addr(exp_avg_scale), _addr(exp_avg_sq_scale), at,
         _HYPER.pack(lr, betas[0], betas[1], eps, weight_decay, int(step)), _addr(grad_scale))
    moved += states
    moved += scales
    _written(moved)


class AdamW:
    """AdamW over a list of parameters, grouped by dtype and device, with f32 or 8-bit states (adamw_step).  steps counts the
    calls of step; a parameter's own steps are those in which it had a gradient (missed, a list a group, counts the others), and
    one without leaves it and its states as they are."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=32):
        if state_bits not in (8, 32):
            raise DetAttnError("state_bits must be 8 or 32")
        params = list(params)
        if len({id(p) for p in params}) != len(params):
            raise DetAttnError("a parameter is given twice: both entries would write it at once")
        self.hyper = dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay)
        self.state_bits, self.steps, self.groups, self.missed = state_bits, 0, [], []
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
            self.missed.append([0] * len(ps))

    def step(self, grad_scale=None):
        self.steps += 1
        for g, missed in zip(self.groups, self.missed):
            ps, grads, none = g["params"], [], 0
            for p in ps:
                x = p.grad
                if x is None:
                    none += 1
                elif not x.is_contiguous():
                    x = x.contiguous()
                grads.append(x)
            if none == len(ps):
                kinds = ()
            elif len(kinds := set(missed)) > 1:
                kinds = sorted({m for m, x in zip(missed, grads) if x is not None})
            with torch.no_grad():
                for m in kinds:   # one launch where all began together
                    adamw_step(ps, grads if len(kinds) == 1 else [x if k == m else None for k, x in zip(missed, grads)], g["exp_avg"],
                               g["exp_avg_sq"], self.steps - m, exp_avg_scale=g.get("exp_avg_scale"),
                               exp_avg_sq_scale=g.get("exp_avg_sq_scale"), grad_scale=grad_scale, **self.hyper)
            if none:
                missed[:] = [k + (x is None) for k, x in zip(missed, grads)]

    def zero_grad(self):
        for g in self.groups:
            for p in g["params"]:
                p.grad = None
