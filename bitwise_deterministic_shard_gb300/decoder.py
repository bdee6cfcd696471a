"""Operators at the ends and in the middle of a decoder: embedding lookup, the gated feed-forward projections and
log probabilities of given tokens with entropy and alternatives, each with its gradient.

Argument marshalling only, as in train.py: the computation runs in the CUDA kernels behind include/detattn.h on the current stream
of the tensors' device, and there is no CPU path.  Every kernel adds in an order that depends on the sizes and types and, for log
probabilities, on where the rows of logits start within 16 bytes, so equal calls (for log probabilities: on equally aligned rows) give
equal bytes on every run.
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple, Optional

import torch

import bitwise_deterministic_shard_gb300 as _da
from bitwise_deterministic_shard_gb300 import DetAttnError
from .train import _HALF, _MATRIX, _addr, _code, _on, _room, _run, _tracked, _written

TOP_MOST = 32         # alternatives of a row in log_probs

_NAMES = ("dgl_forward", "dgl_backward", "dlp_forward", "dlp_backward", "dte_forward", "dte_backward")


def declare(L):
    """Argument types of these entry points of a loaded library."""
    P, I, N, Q = C.c_void_p, C.c_int, C.c_size_t, C.c_int64
    L.dgl_saved_bytes.argtypes, L.dgl_saved_bytes.restype = [Q, Q], N
    L.dgl_workspace_bytes.argtypes, L.dgl_workspace_bytes.restype = [Q, Q], N
    L.dgl_forward.argtypes = [P, P, P, I, P, P, P, P]
    L.dgl_backward.argtypes = [P, P, P, P, P, P, P, P, P, N, P, P]
    L.dlp_forward.argtypes = [P, P, C.c_float, I, P, P, P, P, P, P, P]
    L.dlp_backward.argtypes = [P, P, P, P, P, C.c_float, P, P]
    L.dte_forward.argtypes = [P, I, P, C.c_float, P, P, P]
    L.dte_workspace_bytes.argtypes, L.dte_workspace_bytes.restype = [Q, Q], N
    L.dte_backward.argtypes = [P, I, P, C.c_float, Q, P, P, N, P, P]
    for f in _NAMES:
        getattr(L, f).restype = C.c_int


def _status(status, index):
    if status is None:
        return None
    _on(index, "status", status)
    return _da._sptr(status).value


def _run_of_rows(t, cols):
    """The row stride of t [..., cols] as one run of rows of contiguous columns, or None where there is none."""
    if t.is_contiguous():
        return cols
    if t.dim() < 2 or (cols > 1 and t.stride(-1) != 1):
        return None
    run = want = None       # the leading dimensions, from the last on; those of one entry do not count
    for i in range(t.dim() - 2, -1, -1):
        if t.shape[i] > 1:
            if run is None:
                run = want = t.stride(i)
            if t.stride(i) != want:
                return None
            want *= t.shape[i]
    return cols if run is None else run if run >= cols else None


def _apart(out, *inputs):
    """Refuses a contiguous out that shares memory with an input, given as the bytes of a matrix: other threads may still read what
    one has overwritten."""
    a0, size = out.data_ptr(), out.element_size()
    a1 = a0 + out.numel() * size
    for m in inputs:
        at, _, rows, cols, run = _MATRIX.unpack(m)
        i = max(0, (a0 - at - cols * size) // (run * size) + 1)     # the first row that ends past out's start
        if i < rows and at + i * run * size < a1:
            raise DetAttnError("out must not share memory with the inputs")


# ---------------------------------------------------------------- gated feed-forward

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}


def _tiles(t, code, cols):
    """t [..., cols] as the bytes of a matrix that the kernels can address (16-byte starts and row strides), and t: itself
    or a contiguous copy."""
    run = _run_of_rows(t, cols)
    if run is None or run % 8 or t.data_ptr() % 16:
        t = t.detach().clone(memory_format=torch.contiguous_format)
        run = cols
    return _MATRIX.pack(t.data_ptr(), code, t.numel() // cols, cols, run), t


def _gated_args(x, w_gate, w_up):
    _da._cuda(x, "x")
    dt, index, code = x.dtype, x.get_device(), _HALF.get(x.dtype, 0)
    if not code:
        raise DetAttnError(f"x must be bf16 or f16, not {dt}")
    if x.dim() < 1 or w_gate.dim() != 2 or w_up.shape != w_gate.shape or w_gate.shape[1] != x.shape[-1]:
        raise DetAttnError("x must be [..., width], w_gate and w_up [hidden, width]")
    for t in (w_gate, w_up):
        if t.get_device() != index or t.dtype != dt:
            raise DetAttnError("w_gate and w_up must have x's dtype and device")
    F, D = w_gate.shape
    if D < 8 or F < 8 or D % 8 or F % 8:
        raise DetAttnError("width and hidden must be multiples of 8")
    return index, code, D, F


def gated_linear_forward(x, w_gate, w_up, activation="silu", need_saved=True, out=None, status=None):
    """Gated feed-forward projections: (h, saved), h = act(x w_gate^T) * (x w_up^T).

    x [..., width], w_gate and w_up [hidden, width], all bf16 or all f16, width and hidden multiples of 8; h [..., hidden].
    activation: "silu", "gelu" (with the error function), "gelu_tanh" or "relu" (whose derivative follows the sign of the
    binary32 sum: of a g that is within that sum's rounding of 0, either one).  Both products are binary32 sums, h is
    rounded once.  saved, which the backward pass takes, holds act(g) and act'(g) u rounded to 24 bits each (6 bytes a hidden
    value); None without need_saved.  Up to 16 tokens without it the weights are read once by another kernel, whose sums are in
    another order.  Tensors that the kernels cannot address (columns not contiguous, starts or row strides off 16 bytes) are
    copied.  out must not share memory with the inputs."""
    index, code, D, F = _gated_args(x, w_gate, w_up)
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise DetAttnError(f"activation must be one of {', '.join(ACTIVATIONS)}")
    status = _status(status, index)
    shape, n = (*x.shape[:-1], F), x.numel() // D
    X, x = _tiles(x, code, D)
    G, w_gate = _tiles(w_gate, code, D)
    U, w_up = _tiles(w_up, code, D)
    given = out
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
    else:
        _on(index, "out", out)
        if out.dtype != x.dtype or out.shape != shape or not out.is_contiguous() or out.data_ptr() % 16:
            raise DetAttnError(f"out must be contiguous {x.dtype} {shape} that starts on 16 bytes")
        _apart(out, X, G, U)
    L = _da.lib()
    saved = torch.empty(L.dgl_saved_bytes(n, F), dtype=torch.uint8, device=x.device) if need_saved else None
    _run("gated_linear_forward", index, L.dgl_forward, X, G, U, act, _MATRIX.pack(out.data_ptr(), code, n, F, F), _addr(saved),
         status)
    if given is not None:
        _written(out)
    return out, saved


def gated_linear_backward(grad, x, w_gate, w_up, saved, need_x=True, need_weights=True, workspace=None, status=None):
    """(dx, dw_gate, dw_up) of sum(h * grad) from gated_linear_forward's saved; None where not needed.  The gradients of the two
    products are rounded to x's dtype before the products with the weights and with x."""
    index, code, D, F = _gated_args(x, w_gate, w_up)
    if grad.get_device() != index or grad.dtype != x.dtype or grad.shape != (*x.shape[:-1], F):
        raise DetAttnError(f"grad must be {x.dtype} {(*x.shape[:-1], F)} on x's device")
    n, L, dev, dt = x.numel() // D, _da.lib(), x.device, x.dtype
    if saved is None or saved.get_device() != index or saved.dtype != torch.uint8 or saved.numel() != L.dgl_saved_bytes(n, F) or not saved.is_contiguous():
        raise DetAttnError("saved must be what gated_linear_forward gave for these sizes")
    status = _status(status, index)
    if not need_x and not need_weights:
        return None, None, None
    shape = x.shape
    H, grad = _tiles(grad, code, F)
    X, x = _tiles(x, code, D)
    G, w_gate = _tiles(w_gate, code, D)
    U, w_up = _tiles(w_up, code, D)
    dx = torch.empty(shape, dtype=dt, device=dev) if need_x else None
    dg, du = (torch.empty(F, D, dtype=dt, device=dev) for _ in range(2)) if need_weights else (None, None)
    need = L.dgl_workspace_bytes(n, F)
    ws = _room(need, workspace, dev, index)
    _run("gated_linear_backward", index, L.dgl_backward, H, X, G, U, _addr(saved),
         None if dx is None else _MATRIX.pack(dx.data_ptr(), code, n, D, D),
         None if dg is None else _MATRIX.pack(dg.data_ptr(), code, F, D, D),
         None if du is None else _MATRIX.pack(du.data_ptr(), code, F, D, D), _addr(ws), need, status)
    return dx, dg, du


class _GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation, status):
        h, saved = gated_linear_forward(x, w_gate, w_up, activation, status=status)
        ctx.save_for_backward(x, w_gate, w_up, saved)
        ctx.status = status
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        x, w_gate, w_up, saved = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dg, du = gated_linear_backward(grad, x, w_gate, w_up, saved, need[0], need[1] or need[2], status=ctx.status)
        return dx, dg if need[1] else None, du if need[2] else None, None, None


def gated_linear(x, w_gate, w_up, activation="silu", status=None):
    """gated_linear_forward's h, with autograd for x, w_gate and w_up.  (A backward pass that is captured into a CUDA graph calls
    gated_linear_backward itself, as with attention.)"""
    if _tracked(x, w_gate, w_up):
        return _GatedLinear.apply(x, w_gate, w_up, activation, status)
    return gated_linear_forward(x, w_gate, w_up, activation, need_saved=False, status=status)[0]


# ---------------------------------------------------------------- log probabilities

class LogProbs(NamedTuple):
    """Of each row: log_probs of its given token, entropy, and where asked for its most likely tokens [..., top]."""
    log_probs: torch.Tensor
    entropy: torch.Tensor
    top_log_probs: Optional[torch.Tensor]
    top_indices: Optional[torch.Tensor]


def _rows(t, code, cols):
    """t [..., cols] as the bytes of a matrix, t (itself or a contiguous copy) and the row stride."""
    run = _run_of_rows(t, cols)
    if run is None:
        t, run = t.detach().contiguous(), cols
    return _MATRIX.pack(t.data_ptr(), code, t.numel() // cols, cols, run), t, run


def _logits(logits, targets, temperature):
    _da._cuda(logits, "logits")
    if logits.dim() < 1 or logits.shape[-1] < 1:
        raise DetAttnError("logits must be [..., V] with at least one column")
    code, index = _code(logits, "logits"), logits.get_device()
    if targets.get_device() != index or targets.shape != logits.shape[:-1]:
        raise DetAttnError(f"targets must be {list(logits.shape[:-1])} on the logits' device")
    if targets.dtype != torch.int64:
        if targets.dtype.is_floating_point or targets.dtype.is_complex or targets.dtype == torch.bool:
            raise DetAttnError("targets must be integers")
        targets = targets.to(torch.int64)
    if not 2.0 ** -60 <= temperature <= 2.0 ** 60:
        raise DetAttnError("temperature must be from 2^-60 to 2^60")
    return code, index, targets if targets.is_contiguous() else targets.contiguous()


def log_probs_forward(logits, targets, temperature=1.0, top=0, need_saved=True, status=None):
    """Log probabilities of given tokens, entropies and alternatives: (LogProbs, saved).

    logits [..., V] f32, bf16 or f16; targets [...] integers; temperature from 2^-60 to 2^60.  With z = logits / temperature and lse = log sum exp z:
      log_probs = z[target] - lse (a negative target: no token, 0);  entropy = lse - sum p z
      top_indices, top_log_probs [..., top]: the top largest logits (up to 32) in order, equal ones by their index; None for 0
    Results are f32 (indices int64).  A logit of -inf is a token of probability 0; a row of nothing else has entropy 0 and log
    probabilities of -inf.  saved, which the backward pass takes, is None without need_saved.  How a row's sums are shared out depends on
    the number of rows and on where the row starts within 16 bytes: the same row among others, or in a shifted view, can differ in low
    bits (top_indices do not)."""
    code, index, targets = _logits(logits, targets, temperature)
    shape, V, dev = logits.shape[:-1], logits.shape[-1], logits.device
    if not 0 <= top <= min(TOP_MOST, V):
        raise DetAttnError(f"top must be from 0 to {min(TOP_MOST, V)}")
    status = _status(status, index)
    X, logits, _ = _rows(logits, code, V)
    lp, entropy = (torch.empty(shape, dtype=torch.float32, device=dev) for _ in range(2))
    saved = torch.empty((*shape, 3), dtype=torch.float32, device=dev) if need_saved else None
    top_lp = top_at = None
    if top:
        top_lp = torch.empty((*shape, top), dtype=torch.float32, device=dev)
        top_at = torch.empty((*shape, top), dtype=torch.int64, device=dev)
    _run("log_probs_forward", index, _da.lib().dlp_forward, X, targets.data_ptr(), temperature, top, lp.data_ptr(),
         entropy.data_ptr(), _addr(saved), _addr(top_lp), _addr(top_at), status)
    return LogProbs(lp, entropy, top_lp, top_at), saved


def log_probs_backward(logits, targets, saved, grad, grad_entropy=None, temperature=1.0, out=None):
    """Gradient of sum(grad * log_probs) + sum(grad_entropy * entropy) (f32 [...], either None: zeros) for the logits, rounded once
    to their dtype.  out: contiguous memory for it, the logits themselves or none of theirs; without it the rows of the result
    are as far apart as the logits' are, up to 16 bytes."""
    code, index, targets = _logits(logits, targets, temperature)
    shape, V, n = logits.shape[:-1], logits.shape[-1], targets.numel()
    if saved is None or saved.get_device() != index or saved.dtype != torch.float32 or saved.numel() != 3 * n or not saved.is_contiguous():
        raise DetAttnError("saved must be what log_probs_forward gave for these logits")
    grads = []
    for t, name in ((grad, "grad"), (grad_entropy, "grad_entropy")):
        if t is not None:
            if t.get_device() != index or t.dtype != torch.float32 or t.shape != shape:
                raise DetAttnError(f"{name} must be f32 {list(shape)} on the logits' device")
            t = t if t.is_contiguous() else t.contiguous()
        grads.append(t)
    X, x, run = _rows(logits, code, V)
    if out is None:
        step = V + (run - V) % (16 // logits.element_size())    # rows that start on 16 bytes where the logits' do
        out = torch.empty((*shape, step), dtype=logits.dtype, device=logits.device)
        given, out = None, out if step == V else out[..., :V]
    else:
        _on(index, "out", out)
        if out.dtype != logits.dtype or out.shape != logits.shape or not out.is_contiguous():
            raise DetAttnError(f"out must be contiguous {logits.dtype} {list(logits.shape)}")
        if out.data_ptr() != x.data_ptr() or (run != V and n > 1):
            _apart(out, X)
        given, step = out, V
    _run("log_probs_backward", index, _da.lib().dlp_backward, X, targets.data_ptr(), saved.data_ptr(), _addr(grads[0]),
         _addr(grads[1]), temperature, _MATRIX.pack(out.data_ptr(), code, n, V, step))
    if given is not None:
        _written(given)
    return out


class _LogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, temperature, top, status):
        r, saved = log_probs_forward(logits, targets, temperature, top, status=status)
        ctx.save_for_backward(logits, targets, saved)
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(*(t for t in r[2:] if t is not None))
        return tuple(r)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, grad_entropy, *_):
        logits, targets, saved = ctx.saved_tensors
        if grad is None and grad_entropy is None:
            return None, None, None, None, None
        return log_probs_backward(logits, targets, saved, grad, grad_entropy, ctx.temperature), None, None, None, None


def log_probs(logits, targets, temperature=1.0, top=0, status=None):
    """log_probs_forward's LogProbs, with autograd of log_probs and entropy for the logits (the alternatives have no gradient)."""
    if _tracked(logits):
        return LogProbs(*_LogProbs.apply(logits, targets, temperature, top, status))
    return log_probs_forward(logits, targets, temperature, top, need_saved=False, status=status)[0]


# ---------------------------------------------------------------- embedding

def _ids(ids, index):
    _on(index, "ids", ids)
    if ids.dtype not in (torch.int32, torch.int64):
        raise DetAttnError("ids must be int32 or int64")
    return ids if ids.is_contiguous() else ids.contiguous(), 32 if ids.dtype == torch.int32 else 64


def embedding_forward(ids, weight, scale=1.0, out=None, status=None):
    """Embedding lookup: scale * weight[ids], rounded once (scale 1: the same bits).  ids [...] int32 or int64, weight [rows, cols]
    f32, bf16 or f16; the result is [..., cols] of weight's dtype.  An id outside [0, rows) gives zeros and sets
    STATUS_BAD_TARGET.  out must not share memory with weight."""
    _da._cuda(weight, "weight")
    if weight.dim() != 2 or weight.shape[0] < 1 or weight.shape[1] < 1:
        raise DetAttnError("weight must be [rows, cols] with at least one row and column")
    code, index, cols = _code(weight, "weight"), weight.get_device(), weight.shape[1]
    ids, bits = _ids(ids, index)
    status = _status(status, index)
    W, weight, _ = _rows(weight, code, cols)
    shape, given = (*ids.shape, cols), out
    if out is None:
        out = torch.empty(shape, dtype=weight.dtype, device=weight.device)
    else:
        _on(index, "out", out)
        if out.dtype != weight.dtype or out.shape != shape or not out.is_contiguous():
            raise DetAttnError(f"out must be contiguous {weight.dtype} {list(shape)}")
        _apart(out, W)
    _run("embedding_forward", index, _da.lib().dte_forward, ids.data_ptr(), bits, W, scale,
         _MATRIX.pack(out.data_ptr(), code, ids.numel(), cols, cols), status)
    if given is not None:
        _written(given)
    return out


def embedding_backward(grad, ids, rows, scale=1.0, padding_idx=None, workspace=None, status=None):
    """The gradient [rows, cols] of sum(embedding * grad) for the weight, of grad's dtype: each row the binary32 sum over its own
    tokens, in order and 32 at a time, rounded once; a row's bits depend on its own tokens alone.  Tokens of id padding_idx
    give nothing, nor do those outside [0, rows), which set STATUS_BAD_TARGET."""
    _da._cuda(grad, "grad")
    if grad.dim() < 1 or grad.shape[:-1] != ids.shape or grad.shape[-1] < 1:
        raise DetAttnError("grad must be [..., cols] with ids [...]")
    code, index, cols = _code(grad, "grad"), grad.get_device(), grad.shape[-1]
    ids, bits = _ids(ids, index)
    if rows < 1 or (padding_idx is not None and not 0 <= padding_idx < rows):
        raise DetAttnError("rows must be at least 1, padding_idx None or from 0 to rows - 1")
    status = _status(status, index)
    G, grad, _ = _rows(grad, code, cols)
    dw = torch.empty(rows, cols, dtype=grad.dtype, device=grad.device)
    L = _da.lib()
    need = L.dte_workspace_bytes(ids.numel(), cols)
    ws = _room(need, workspace, grad.device, index)
    _run("embedding_backward", index, L.dte_backward, ids.data_ptr(), bits, G, scale, -1 if padding_idx is None else padding_idx,
         _MATRIX.pack(dw.data_ptr(), code, rows, cols, cols), _addr(ws), need, status)
    return dw


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, weight, scale, padding_idx, status):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale, ctx.padding_idx, ctx.status = weight.shape[0], scale, padding_idx, status
        return embedding_forward(ids, weight, scale, status=status)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        ids, = ctx.saved_tensors
        return None, embedding_backward(grad, ids, ctx.rows, ctx.scale, ctx.padding_idx, status=ctx.status), None, None, None


def embedding(ids, weight, scale=1.0, padding_idx=None, status=None):
    """embedding_forward's lookup, with autograd for weight (tokens of id padding_idx give it no gradient)."""
    if padding_idx is not None and not 0 <= padding_idx < weight.shape[0]:
        raise DetAttnError("padding_idx must be None or from 0 to rows - 1")
    if _tracked(weight):
        return _Embedding.apply(ids, weight, scale, padding_idx, status)
    return embedding_forward(ids, weight, scale, status=status)
