"""Operators at the ends and in the middle of a decoder: the gated feed-forward projections, each with its gradient.

Argument marshalling only, as in train.py: the computation runs in the CUDA kernels behind include/detattn.h on the current stream
of the tensors' device, and there is no CPU path.  Every kernel adds in an order that depends on the sizes and types alone,
so equal calls give equal bytes on every run.
"""
from __future__ import annotations

import ctypes as C

import torch

import bitwise_deterministic_shard_gb300 as _da
from bitwise_deterministic_shard_gb300 import DetAttnError
from .train import _HALF, _MATRIX, _addr, _on, _room, _run, _tracked, _written

_NAMES = ("dgl_forward", "dgl_backward")


def declare(L):
    """Argument types of these entry points of a loaded library."""
    P, I, N, Q = C.c_void_p, C.c_int, C.c_size_t, C.c_int64
    L.dgl_saved_bytes.argtypes, L.dgl_saved_bytes.restype = [Q, Q], N
    L.dgl_workspace_bytes.argtypes, L.dgl_workspace_bytes.restype = [Q, Q], N
    L.dgl_forward.argtypes = [P, P, P, I, P, P, P, P]
    L.dgl_backward.argtypes = [P, P, P, P, P, P, P, P, P, N, P, P]
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
    activation: "silu", "gelu" (with the error function), "gelu_tanh" or "relu".  Both products are binary32 sums, h is
    rounded once.  saved, which the backward pass takes, holds act(g) and act'(g) u with 24 bits each (6 bytes a hidden
    value); None without need_saved.  Up to 8 tokens without it the weights are read once by another kernel, whose sums are in
    another order.  Tensors that the kernels cannot address (columns not contiguous, starts or row strides off 16 bytes) are
    copied."""
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
    if saved.get_device() != index or saved.dtype != torch.uint8 or saved.numel() != 6 * n * F or not saved.is_contiguous():
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
