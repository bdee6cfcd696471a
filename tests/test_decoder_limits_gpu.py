"""The decoder's operators at their limits: results of a few bytes, logits as far apart as their type allows, factors beside a
rounding, rows of which little is finite, and two calls at once on new inputs."""
import ctypes
import os
import sys

import pytest
import torch

import bitwise_deterministic_shard_gb300 as da

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import decoder_reference as R  # noqa: E402
import test_decoder_gpu as T  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

TYPES, INF = T.TYPES, float("inf")


def _matrix(t, rows, cols):
    m = da._Matrix()
    m.ptr, m.rows, m.cols, m.row_stride = t.data_ptr(), rows, cols, cols
    m.dtype = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[t.dtype]
    return ctypes.byref(m)


# ---------------------------------------------------------------- embedding

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [0, 1, 4096, 4097, 5000, 32768, 32769, 40000])
def test_every_row_of_a_small_gradient_is_written(n, dtype):
    """Tables of a few bytes, whose zeros are less than a launch's parts of them, from any start: no token gives a gradient (all are
    padding, or unknown), or the last row's alone do.  What lies around the result stays as it was."""
    L, s = da.lib(), torch.cuda.current_stream().cuda_stream
    for rows, cols in ((1, 1), (1, 2), (2, 1), (1, 3), (3, 1), (1, 5), (1, 8), (2, 9), (600, 1)):
        ws = torch.empty(max(1, L.dte_workspace_bytes(n, cols)), dtype=torch.uint8, device="cuda")
        dy = torch.ones(n, cols, device="cuda", dtype=dtype)
        for id_, padding in ((rows - 1, rows - 1), (-1, -1), (rows, -1), (rows - 1, -1)):
            ids = torch.full((n,), id_, device="cuda")
            for start in (8, 9, 11):
                buffer = torch.full((start + rows * cols + 8,), 7.0, device="cuda", dtype=dtype)
                dw = buffer[start:start + rows * cols]
                assert L.dte_backward(ids.data_ptr(), 64, _matrix(dy, n, cols), 1.0, padding, _matrix(dw, rows, cols), ws.data_ptr(),
                                      ws.numel(), None, s) == 0
                want = torch.zeros(rows, cols, device="cuda", dtype=dtype)
                if id_ == rows - 1 and padding < 0:
                    want[-1] = torch.tensor(float(n)).to(dtype)       # ones: every sum is exact
                assert torch.equal(dw.view(rows, cols), want), (rows, cols, id_, padding, start)
                assert (buffer[:start] == 7).all() and (buffer[start + rows * cols:] == 7).all()


# ---------------------------------------------------------------- log probabilities

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows, V, top", [(3, 2, 2), (5, 50, 32), (300, 3001, 20), (4, 40001, 32), (1300, 20000, 5)])
@pytest.mark.parametrize("temperature", [4.0, 1.0e3, 2.0 ** 60])
def test_log_probs_of_logits_farther_apart_than_the_type_reaches(temperature, rows, V, top, dtype):
    """Differences past the largest finite number whose quotients by the temperature are finite: the lowest logits as targets and among
    the alternatives."""
    x, t, a, b = T._logits(rows, V, dtype, 11)
    x[:, 0], x[:, V // 2], x[:, V - 1] = 3e38, -3e38, torch.finfo(dtype).min
    t[0::3], t[1::3], t[2::3] = V // 2, V - 1, 0
    x[1::2, 1:] = torch.where(torch.rand(x[1::2, 1:].shape, device="cuda", generator=T._gen(V)) < 0.5, -3e38, -1.5e38).to(dtype)
    r, _ = T._probs_check(x, t, temperature, top, a, b)
    assert torch.isfinite(r.log_probs).all() and torch.isfinite(r.top_log_probs).all()
    assert (r.log_probs[0] < -5e38 / temperature) and (r.log_probs[1] < -4e38 / temperature)


def test_log_probs_past_the_results_range_are_infinite():
    """Quotients that binary32 does not hold, and those it just holds."""
    x = torch.tensor([[3e38, -3e38, 1.0, -INF]] * 3, device="cuda")
    t = torch.tensor([1, 2, 3], device="cuda")
    for temperature in (0.5, 1.0, 1.7, 1.8, 2.0):
        r = da.log_probs_forward(x, t, temperature, 4)[0]
        want = R.log_probs(x, t, torch.tensor(temperature).item(), 4)
        for got, w in ((r.log_probs, want["lp"]), (r.top_log_probs, want["top_lp"])):
            T._close(got, w.float().double(), 1.02 * 5 * R.e * w.abs() + 1e-30, temperature)
        assert torch.equal(r.top_indices, want["top"]) and (r.entropy == 0).all()
        assert r.log_probs[0].isinf() == (temperature < 1.75) and r.log_probs[1].isinf() == (temperature < 0.8) and r.log_probs[2] == -INF


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, V", [(5, 40001), (300, 3001), (1300, 20003)])
def test_log_probs_have_equal_bytes_in_equally_aligned_places(rows, V, dtype):
    """The order of a row's sums depends on the number of rows and on where the rows start within 16 bytes: on nothing else of
    their place.  Other starts and other numbers of rows stay within the tolerance of the sums."""
    per = 16 // dtype.itemsize
    x, t, a, b = T._logits(rows, V, dtype, 12)
    want, dx = T._probs_check(x, t, 0.9, 7, a, b)
    buffer = torch.empty(rows * V + 3 * per, device="cuda", dtype=dtype)
    same = buffer[2 * per:2 * per + rows * V].view(rows, V)
    wide = torch.empty(rows, V + 5 * per, device="cuda", dtype=dtype)[:, :V]      # rows that start as x's do
    other = torch.empty(rows, V + 5 * per + 3, device="cuda", dtype=dtype)[:, 1:V + 1]
    for y, equal in ((same, True), (wide, True), (other, False)):
        y.copy_(x)
        got, grad = T._probs_check(y, t, 0.9, 7, a, b)
        assert torch.equal(got.top_indices, want.top_indices)
        if equal:
            assert all(torch.equal(p, q) for p, q in zip(got, want)) and torch.equal(grad, dx)
    first, _ = T._probs_check(x[:1], t[:1], 0.9, 7, a[:1], b[:1])      # a row by itself
    assert torch.equal(first.top_indices, want.top_indices[:1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [70, 3000, 40001, 128256])
def test_alternatives_of_rows_of_which_little_is_finite(V, dtype):
    """Finite logits at every other place; fewer than the alternatives, spread over the row, at its ends, side by side; among the type's
    lowest; none: the finite ones come first in order, then the first of the others."""
    g, places = T._gen(V), torch.arange(V, device="cuda")
    up = (places.float() / V * 8).to(dtype)
    nothing = torch.full_like(up, -INF)
    x = [torch.where(places % 2 == 1, up, nothing), torch.where(places % 2 == 0, -up, nothing)]
    for k in (1, 2, 5, 31, 32, 33):
        row = nothing.clone()
        row[torch.randperm(V, device="cuda", generator=g)[:k]] = T._randn(k, g=g, to=dtype)
        x.append(row)
    for at in ([0], [V - 1], [0, V - 1], list(range(V - 9, V)), list(range(20))):
        row = nothing.clone()
        row[at] = 1.5
        x.append(row)
    low = torch.where(places % 3 == 0, torch.full_like(up, torch.finfo(dtype).min), nothing)
    x.append(low.clone())
    low[V // 2] = 3.0
    x += [low, nothing]
    x = torch.stack(x)
    t = torch.zeros(len(x), dtype=torch.int64, device="cuda")
    for top in (1, 3, 8, 20, 32):
        r = da.log_probs_forward(x, t, 1.0, top)[0]
        want = torch.sort(x, dim=1, descending=True, stable=True)
        assert torch.equal(r.top_indices, want.indices[:, :top]), top
        assert torch.equal(r.top_log_probs == -INF, want.values[:, :top] == -INF), top


# ---------------------------------------------------------------- gated feed-forward

@pytest.mark.parametrize("dtype, bits", [(torch.bfloat16, 8), (torch.float16, 11)])
@pytest.mark.parametrize("tokens", [1, 300])
def test_gated_factors_are_rounded_to_nearest(tokens, dtype, bits):
    """A factor v is kept with 16 significant bits and rounded to the operands' type in the backward pass.  Here v is half a step of that type above 1,
    and three quarters of a step of 2^-15 more: to nearest this stays above the half step and the gradient is rounded up;
    cut off toward zero it falls back onto the half step, which goes to the even neighbour, 1."""
    x = torch.zeros(tokens, 16, device="cuda", dtype=dtype)
    half, step = 2.0 ** -bits, 2.0 ** (1 - bits)
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 1.0, half, 2.0 ** -9, 2.0 ** -9
    wg, wu = (torch.zeros(24, 16, device="cuda", dtype=dtype) for _ in range(2))
    sign = torch.where(torch.arange(24, device="cuda") % 3 == 0, -1.0, 1.0).to(dtype)
    for w, s in ((wg, torch.ones_like(sign)), (wu, sign)):            # relu: q = g, p = u
        w[:, 0], w[:, 1], w[:, 2], w[:, 3] = s, s, s * 2.0 ** -7, s * 2.0 ** -8
    h, saved = da.gated_linear_forward(x, wg, wu, "relu")
    dh = torch.zeros(tokens, 24, device="cuda", dtype=dtype)
    dh[0] = 1.0
    _, dwg, dwu = da.gated_linear_backward(dh, x, wg, wu, saved)      # one token: dwu[:, 0] = du x[0, 0] = q
    v = 1.0 + half + 2.0 ** -16 + 2.0 ** -17
    assert torch.tensor(v, dtype=torch.float64).to(dtype) == 1 + step
    assert (dwu[:, 0] == 1 + step).all() and torch.equal(dwg[:, 0], (1 + step) * sign)


def test_gated_factors_at_the_ends_of_binary32():
    """The largest finite factor stays finite, infinities and NaN stay what they are."""
    t, top, far = torch.bfloat16, 2.0 - 2.0 ** -7, 2.0 ** 120
    x = torch.zeros(4, 16, device="cuda", dtype=t)
    x[:, :4] = 1.0
    x[2, 5], x[3, 5] = INF, float("nan")
    wg, wu = (torch.zeros(24, 16, device="cuda", dtype=t) for _ in range(2))
    wg[:, 3], wg[:, 5] = 1.0, 1.0
    wu[:, 0], wu[:, 1], wu[:, 2] = top * 2.0 ** 127, top * 2.0 ** 119, top * 2.0 ** 111      # their sum is 2^128 - 2^104
    wu[1::2] = -wu[1::2]
    h, saved = da.gated_linear_forward(x, wg, wu, "relu")
    dh = torch.zeros(4, 24, device="cuda", dtype=t)
    for row, want in ((0, far), (1, far), (2, INF), (3, float("nan"))):
        dh.zero_()
        dh[row] = 2.0 ** -8
        _, dwg, dwu = da.gated_linear_backward(dh[row:row + 1], x[row:row + 1], wg, wu, da.gated_linear_forward(x[row:row + 1], wg, wu, "relu")[1])
        if row < 2:
            assert (dwg[0::2, 3] == want).all() and (dwg[1::2, 3] == -want).all() and (dwu[:, 3] == 2.0 ** -8).all()
        elif row == 2:
            assert (dwu[:, 3] == INF).all()
        else:
            assert dwu[:, 3].isnan().all()


# ---------------------------------------------------------------- graphs and streams

def _replayed_and_at_once(sets, step):
    """step(*set) captured twice, both graphs replayed on two streams with other inputs each time, and called on two streams
    at once: equal bytes to a call alone."""
    want = [[v.clone() for v in step(*s)] for s in sets]
    held = [[v.clone() for v in sets[i]] for i in range(2)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for h in held:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(step(*h))
    for turn in range(3):
        for k in range(2):
            for to, new in zip(held[k], sets[(turn + k) % len(sets)]):
                to.copy_(new)
        torch.cuda.synchronize()
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(p, q) for p, q in zip(outs[k], want[(turn + k) % len(sets)]))
    got = []
    for i, s in enumerate(sets):
        with torch.cuda.stream(streams[i % 2]):
            got.append(step(*s))
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert all(torch.equal(v, w) for v, w in zip(p, q))


@pytest.mark.parametrize("tokens, D, F, dtype", [(1, 520, 1000, torch.bfloat16), (13, 2048, 4104, torch.float16), (48, 264, 1032, torch.float16),
                                                 (700, 520, 1000, torch.bfloat16), (2049, 1000, 2744, torch.float16)])
def test_gated_in_graphs_and_on_two_streams(tokens, D, F, dtype):
    sets = [T._gated_inputs(tokens, D, F, dtype, seed) for seed in range(20, 24)]

    def step(x, wg, wu, dh):
        h, saved = da.gated_linear_forward(x, wg, wu, "gelu")
        return (h, *da.gated_linear_backward(dh, x, wg, wu, saved), da.gated_linear(x, wg, wu))
    _replayed_and_at_once(sets, step)


@pytest.mark.parametrize("rows, V, top, dtype", [(1, 128256, 32, torch.float32), (8, 70001, 20, torch.bfloat16), (100, 16385, 5, torch.float16),
                                                 (300, 3001, 7, torch.float32), (1300, 20000, 3, torch.bfloat16), (3000, 200, 0, torch.float16)])
def test_log_probs_in_graphs_and_on_two_streams(rows, V, top, dtype):
    sets = [T._logits(rows, V, dtype, seed) for seed in range(30, 34)]

    def step(x, t, a, b):
        r, saved = da.log_probs_forward(x, t, 1.1, top)
        return (*(v for v in r if v is not None), da.log_probs_backward(x, t, saved, a, b, 1.1))
    _replayed_and_at_once(sets, step)
