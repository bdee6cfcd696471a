"""The decoder's operators on the GPU against plain 64-bit forms, at the sizes, masks, strides and types where they can go wrong."""
import ctypes
import math
import os
import sys

import pytest
import torch

import bitwise_deterministic_shard_gb300 as da

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import decoder_reference as R  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

TYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")


def _close(got, want, tol, what):
    same = got.double() == want                          # infinities
    d = (got.double() - want).abs()
    bad = ~((d <= tol) | same)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {d.numel()} outside, worst {float((d / tol).nan_to_num(9e9).max())} of the tolerance"


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(*shape, g, to=torch.float32, by=1.0):
    return (torch.randn(*shape, device="cuda", generator=g) * by).to(to)


# ---------------------------------------------------------------- embedding

def _words(n, v, g):
    """A few ids often, most of them rarely."""
    return (torch.rand(n, device="cuda", generator=g, dtype=torch.float64) ** 4 * v).long().clamp_(0, v - 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n, v, w", [(0, 5, 8), (1, 1, 1), (5, 20, 16), (32, 1, 8), (33, 1, 33), (64, 1, 8), (65, 1, 33), (129, 3, 264), (3001, 2001, 1003),
                                     (4096, 5000, 72), (4097, 5000, 72), (16385, 70001, 40), (40000, 513, 136), (9000, 2, 24), (20000, 262145, 8),
                                     (33000, 1, 8), (5000, 1, 40)])
def test_embedding(n, v, w, dtype):
    """Rows of no, one, 32, 33 and thousands of tokens; one CTA's sort and the longer one; one to three digits."""
    g = _gen(n + v)
    ids, weight, dy = _words(n, v, g), _randn(v, w, g=g, to=dtype), _randn(n, w, g=g, to=dtype)
    st = da.new_status()
    for scale, padding, kind in ((1.0, None, torch.int64), (1.7, 0, torch.int32)):
        y = da.embedding_forward(ids.to(kind), weight, scale, status=st)
        dw = da.embedding_backward(dy, ids.to(kind), v, scale, padding, status=st)
        r = R.embedding(ids, weight, dy, scale, padding)
        tol = R.embedding_tolerance(r, dtype, scale)
        _close(y, r["y"], tol["y"], "y")
        _close(dw, r["dw"], tol["dw"], "dw")
        if padding is not None:
            assert (dw[0] == 0).all()
        assert (dw[r["count"] == 0] == 0).all()
    assert da.read_status(st) == 0


@pytest.mark.parametrize("n, v", [(32768, 600), (32769, 300000), (131072, 5), (131073, 5), (150001, 70000), (200000, 1)])
def test_embedding_of_many_tokens(n, v):
    """The longer sort's blocks of both sizes, up to 32 of them and more."""
    g = _gen(n)
    ids, dy = _words(n, v, g), _randn(n, 12, g=g)
    dw = da.embedding_backward(dy, ids, v)
    r = R.embedding(ids, torch.zeros(v, 12, device="cuda"), dy)
    _close(dw, r["dw"], R.embedding_tolerance(r, torch.float32, 1.0)["dw"], "dw")
    assert torch.equal(dw, da.embedding_backward(dy, ids.int(), v))


@pytest.mark.parametrize("n", [50, 20000])
def test_embedding_unknown_ids(n):
    g = _gen(1)
    ids, weight, dy = _words(n, 40, g), _randn(40, 24, g=g), _randn(n, 24, g=g)
    ids[::7], ids[::11], ids[3] = -1, 40, 2 ** 40
    st = da.new_status()
    y = da.embedding_forward(ids, weight, status=st)
    assert da.read_status(st) == da.STATUS_BAD_TARGET
    st.zero_()
    dw = da.embedding_backward(dy, ids, 40, status=st)
    assert da.read_status(st) == da.STATUS_BAD_TARGET
    r = R.embedding(ids, weight, dy)
    tol = R.embedding_tolerance(r, torch.float32, 1.0)
    _close(y, r["y"], tol["y"], "y")
    _close(dw, r["dw"], tol["dw"], "dw")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["batch", "slice", "odd", "broadcast", "columns"])
def test_embedding_layouts(layout, dtype):
    g = _gen(2)
    ids = _words(600, 90, g).view(20, 30)
    w, dy = _randn(90, 64, g=g, to=dtype), _randn(20, 30, 64, g=g, to=dtype)
    if layout == "slice":                                # rows of a wider buffer that start on 16 bytes
        w, dy = _randn(90, 96, g=g, to=dtype)[:, 16:80], _randn(20, 30, 80, g=g, to=dtype)[..., :64]
    if layout == "odd":
        w, dy = _randn(90, 67, g=g, to=dtype)[:, 1:65], _randn(20, 30, 67, g=g, to=dtype)[..., 3:]
    if layout == "broadcast":
        dy = _randn(64, g=g, to=dtype).expand(20, 30, 64)
    if layout == "columns":
        w, dy, ids = _randn(64, 90, g=g, to=dtype).T, _randn(30, 20, 64, g=g, to=dtype).transpose(0, 1), ids.T.contiguous().T
    r = R.embedding(ids, w, dy, 0.5)
    tol = R.embedding_tolerance(r, dtype, 0.5)
    _close(da.embedding_forward(ids, w, 0.5), r["y"], tol["y"], "y")
    _close(da.embedding_backward(dy, ids, 90, 0.5), r["dw"], tol["dw"], "dw")
    weight = w.detach().requires_grad_(True)
    out = da.embedding(ids, weight, 0.5)
    out.backward(dy)
    assert torch.equal(weight.grad, da.embedding_backward(dy, ids, 90, 0.5)) and torch.equal(out, da.embedding_forward(ids, w, 0.5))


def test_embedding_keeps_bits_and_special_values():
    """A scale of 1 copies bits; NaN and infinities stay in their own rows."""
    w = torch.randint(0, 1 << 16, (300, 40), device="cuda").to(torch.int16).view(torch.bfloat16)
    ids = torch.randint(0, 300, (500,), device="cuda")
    assert torch.equal(da.embedding_forward(ids, w).view(torch.int16), w[ids].view(torch.int16))
    dy = torch.ones(500, 40, device="cuda")
    dy[7], dy[9, 3] = float("nan"), INF
    dw = da.embedding_backward(dy, torch.arange(500, device="cuda") % 250, 300)
    assert dw[7].isnan().all() and dw[9, 3] == INF and torch.isfinite(dw[[0, 8, 10, 299]]).all() and (dw[9, :3] == 2).all()


def test_embedding_row_depends_on_its_own_tokens():
    """A row's gradient has the same bits whatever the other tokens are, and on every run."""
    g = _gen(3)
    for n in (7000, 30000):
        ids, dy = torch.randint(0, 50, (n,), device="cuda", generator=g), _randn(n, 72, g=g)
        first = da.embedding_backward(dy, ids, 50)
        assert torch.equal(first, da.embedding_backward(dy, ids, 50))
        other = torch.where(ids == 17, 17, torch.randint(18, 4000, (n,), device="cuda", generator=g))
        assert torch.equal(first[17], da.embedding_backward(dy, other, 4000)[17])


@pytest.mark.parametrize("n, v, w", [(20, 300, 16), (3000, 20000, 264), (20000, 70000, 136), (40000, 900, 33)])
def test_embedding_in_graphs_and_on_two_streams(n, v, w):
    """Replayed with other ids and gradients, and two calls at once: equal bytes to a call alone."""
    g = _gen(n + w)
    sets = [(_words(n, v, g), _randn(n, w, g=g, to=torch.bfloat16)) for _ in range(4)]
    weight = _randn(v, w, g=g, to=torch.bfloat16)
    want = [(da.embedding_forward(ids, weight, 2.0), da.embedding_backward(dy, ids, v, 2.0, 0)) for ids, dy in sets]
    held = [[t.clone() for t in sets[i]] for i in range(2)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for ids, dy in held:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append((da.embedding_forward(ids, weight, 2.0), da.embedding_backward(dy, ids, v, 2.0, 0)))
    for turn in range(3):
        for k in range(2):
            for to, new in zip(held[k], sets[(turn + k) % 4]):
                to.copy_(new)
        torch.cuda.synchronize()
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            assert all(torch.equal(p, q) for p, q in zip(outs[k], want[(turn + k) % 4]))
    got = [[], []]
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            got[i % 2].append(da.embedding_backward(sets[i][1], sets[i][0], v, 2.0, 0))
    torch.cuda.synchronize()
    assert all(torch.equal(got[i % 2][i // 2], want[i][1]) for i in range(4))


def test_embedding_offsets_past_32_bits():
    v, w = 530000, 4104                                   # 2.17e9 elements
    weight = torch.zeros(v, w, device="cuda", dtype=torch.bfloat16)
    weight[-1], weight[v // 2] = 3.0, 5.0
    ids = torch.tensor([v - 1, 0, v // 2, v - 1], device="cuda")
    y = da.embedding_forward(ids, weight)
    assert (y[0] == 3).all() and (y[1] == 0).all() and (y[2] == 5).all()
    del weight
    dw = da.embedding_backward(torch.ones(4, w, device="cuda", dtype=torch.bfloat16), ids, v)
    assert (dw[-1] == 2).all() and (dw[v // 2] == 1).all() and (dw[0] == 1).all() and int(dw.count_nonzero()) == 3 * w
    del dw
    n = 530000
    ids = torch.zeros(n, device="cuda", dtype=torch.int64)
    ids[-1] = 1
    y = da.embedding_forward(ids, torch.tensor([[1.0] * w, [2.0] * w], device="cuda", dtype=torch.bfloat16))
    assert (y[-1] == 2).all() and (y[-2] == 1).all()
    dw = da.embedding_backward(y, ids, 2)
    assert (dw[1] == 2).all() and (dw[0] == torch.tensor(n - 1.0).to(torch.bfloat16).cuda()).all()


# ---------------------------------------------------------------- gated feed-forward

def _gated_inputs(T, D, F, dtype, seed=0, by=None):
    g = _gen(seed + T + D + F)
    by = D ** -0.5 if by is None else by
    return _randn(T, D, g=g, to=dtype), _randn(F, D, g=g, to=dtype, by=by), _randn(F, D, g=g, to=dtype, by=by), _randn(T, F, g=g, to=dtype)


def _gated_check(x, wg, wu, dh, kind):
    st = da.new_status()
    h, saved = da.gated_linear_forward(x, wg, wu, kind, status=st)
    grads = da.gated_linear_backward(dh, x, wg, wu, saved, status=st)
    assert da.read_status(st) == 0
    r = R.gated(x.reshape(-1, x.shape[-1]), wg, wu, dh.reshape(-1, dh.shape[-1]), kind)
    tol = R.gated_tolerance(r, x.dtype, kind)
    for got, n in zip((h, *grads), ("h", "dx", "dwg", "dwu")):
        _close(got.reshape(r[n].shape), r[n], tol[n], n)
        if r[n].numel() > 10000:                          # rounded once, the gradients' factors once more: u / sqrt(3) each at most
            off, u = float((got.double().reshape(r[n].shape) - r[n]).norm() / r[n].norm()), R.half_step(x.dtype)
            assert off <= (0.6 if n == "h" else 0.85) * u, f"{n}: {off / u} half steps in the mean"
    few = da.gated_linear(x, wg, wu, kind)
    _close(few.reshape(r["h"].shape), r["h"], tol["h"], "h without saved")
    return h, saved, grads


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T, D, F", [(1, 8, 8), (2, 64, 40), (3, 72, 136), (7, 520, 24), (8, 1000, 248), (9, 8, 16), (31, 264, 128), (128, 64, 64),
                                     (129, 200, 72), (256, 128, 256), (257, 136, 264), (300, 1000, 520), (777, 312, 2744), (2049, 72, 1032)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated(T, D, F, dtype, kind):
    _gated_check(*_gated_inputs(T, D, F, dtype), kind)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("T", [3, 5, 200])
def test_gated_activations(T, kind, dtype):
    """Products of every size: far into both tails, and around zero."""
    _gated_check(*_gated_inputs(T, 256, 344, dtype, 1, by=0.5), kind)
    x, wg, wu, dh = _gated_inputs(T, 256, 344, dtype, 2)
    wg[:40] = 0                                            # act(0)
    _gated_check(x, wg, wu, dh, kind)


@pytest.mark.parametrize("T, D, F", [(4000, 520, 5000), (600, 2048, 10008), (20000, 72, 264), (100, 4104, 12296), (5000, 1544, 1400)])
def test_gated_many_tiles(T, D, F):
    """More tiles than pairs of SMs, wide and narrow ones, in rounds that do not come out even."""
    _gated_check(*_gated_inputs(T, D, F, torch.bfloat16, 3), "silu")


@pytest.mark.parametrize("layout", ["batch", "slice", "odd", "fused", "broadcast", "columns"])
@pytest.mark.parametrize("T", [4, 60])
def test_gated_layouts(layout, T):
    g, t = _gen(4), torch.bfloat16
    x, wg, wu, dh = _gated_inputs(T, 64, 96, t, 4)
    if layout == "batch":
        x, dh = x.view(2, T // 2, 64), dh.view(2, T // 2, 96)
    if layout == "slice":
        x, wg, dh = _randn(T, 80, g=g, to=t)[:, 8:72], _randn(96, 72, g=g, to=t, by=0.1)[:, :64], _randn(T, 128, g=g, to=t)[:, 32:]
    if layout == "odd":
        x, wu, dh = _randn(T, 67, g=g, to=t)[:, 1:65], _randn(96, 68, g=g, to=t, by=0.1)[:, 2:66], _randn(T, 97, g=g, to=t)[:, 1:]
    if layout == "fused":                                  # both weights in one tensor
        wg, wu = (_randn(192, 64, g=g, to=t, by=0.1)).split(96)
    if layout == "broadcast":
        x, dh = x[:1].expand(T, 64), dh[:1].expand(T, 96)
    if layout == "columns":
        x, wg, dh = _randn(64, T, g=g, to=t).T, _randn(64, 96, g=g, to=t, by=0.1).T, _randn(96, T, g=g, to=t).T
    _gated_check(x, wg, wu, dh, "silu")
    leaves = [v.detach().requires_grad_(True) for v in (x, wg, wu)]
    h = da.gated_linear(*leaves)
    h.backward(dh)
    want, saved = da.gated_linear_forward(x, wg, wu)
    assert torch.equal(h, want)
    for leaf, got in zip(leaves, da.gated_linear_backward(dh, x, wg, wu, saved)):
        assert torch.equal(leaf.grad, got)


def test_gated_parts_alone_and_none():
    x, wg, wu, dh = _gated_inputs(300, 72, 136, torch.float16, 5)
    h, saved = da.gated_linear_forward(x, wg, wu)
    all_ = da.gated_linear_backward(dh, x, wg, wu, saved)
    dx, a, b = da.gated_linear_backward(dh, x, wg, wu, saved, need_weights=False)
    assert torch.equal(dx, all_[0]) and a is None and b is None
    dx, a, b = da.gated_linear_backward(dh, x, wg, wu, saved, need_x=False)
    assert dx is None and torch.equal(a, all_[1]) and torch.equal(b, all_[2])
    assert da.gated_linear_backward(dh, x, wg, wu, saved, False, False) == (None, None, None)
    h, saved = da.gated_linear_forward(x[:0], wg, wu)
    dx, a, b = da.gated_linear_backward(dh[:0], x[:0], wg, wu, saved)
    assert h.shape == (0, 136) and dx.shape == (0, 72) and (a == 0).all() and (b == 0).all()
    assert da.gated_linear(x[0], wg, wu).shape == (136,)


@pytest.mark.parametrize("D, F", [(264, 1032), (2048, 10008)])
def test_gated_rows_do_not_depend_on_the_batch(D, F):
    """A token's h and dx have the same bits with any other tokens, in wide tiles and narrow ones; up to 16 tokens without saved
    factors among themselves."""
    x, wg, wu, dh = _gated_inputs(4000, D, F, torch.bfloat16, 9)
    h, saved = da.gated_linear_forward(x, wg, wu)
    dx = da.gated_linear_backward(dh, x, wg, wu, saved, need_weights=False)[0]
    for n in (1, 5, 17, 300, 2100):
        some, part = da.gated_linear_forward(x[:n], wg, wu)
        assert torch.equal(some, h[:n])
        assert torch.equal(da.gated_linear_backward(dh[:n], x[:n], wg, wu, part, need_weights=False)[0], dx[:n])
        alone = da.gated_linear(x[:n], wg, wu)
        assert torch.equal(alone, h[:n] if n > 16 else da.gated_linear(x[:16], wg, wu)[:n])


def test_gated_special_values_stay_in_their_rows():
    """A row of NaN or infinities gives what the formula gives there, and nothing elsewhere."""
    for T in (6, 300):
        x, wg, wu, dh = _gated_inputs(T, 64, 96, torch.bfloat16, 6)
        want = da.gated_linear(x, wg, wu)
        x[2], x[4] = float("nan"), 1e30
        got = da.gated_linear(x, wg, wu)
        assert got[2].isnan().all()
        keep = torch.ones(T, dtype=torch.bool, device="cuda")
        keep[[2, 4]] = False
        assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("power", [7, 50, 62])
def test_gated_far_activations(power, kind):
    """Where act' is 0 or 1 and the cubic, the square or the exponential overflow: powers of two, so every result is exact."""
    far = 2.0 ** power
    x = torch.zeros(3, 8, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[0, 1], x[2, 0], x[2, 1] = far, 1.0, -far, 1.0
    wg, wu = torch.zeros(2, 16, 8, dtype=torch.bfloat16, device="cuda").unbind(0)
    wg[:, 0], wu[:, 1] = 1.0, 2.0
    dh = torch.full((3, 16), 0.5, dtype=torch.bfloat16, device="cuda")
    h, saved = da.gated_linear_forward(x, wg, wu, kind)
    dx, dwg, dwu = da.gated_linear_backward(dh, x, wg, wu, saved)
    for got in (h, da.gated_linear(x, wg, wu, kind)):
        assert (got[0] == 2 * far).all() and (got[1:] == 0).all()
    want = torch.zeros(3, 8, device="cuda")
    want[0, 0], want[0, 1] = 16.0, 16 * far                # sums over the 16 hidden units of dh u and 2 dh act(g)
    assert torch.equal(dx.float(), want)
    assert (dwg[:, 0] == far).all() and (dwg[:, 1] == 1).all() and (dwg[:, 2:] == 0).all()
    assert (dwu[:, 0] == far * far / 2).all() and (dwu[:, 1] == far / 2).all() and (dwu[:, 2:] == 0).all()


def test_gated_same_bytes_on_another_stream_and_in_a_graph():
    x, wg, wu, dh = _gated_inputs(700, 520, 1000, torch.bfloat16, 7)

    def step():
        h, saved = da.gated_linear_forward(x, wg, wu)
        return (h, *da.gated_linear_backward(dh, x, wg, wu, saved), da.gated_linear(x[:3], wg, wu))
    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graphs = []
    for _ in range(2):                                     # two graphs, replayed by turns
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, step()))
    for _ in range(3):
        for graph, out in graphs:
            for t in out:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_gated_offsets_past_32_bits():
    T, D, F = 66000, 64, 32776                             # 2.16e9 hidden values
    x, wg, wu, _ = _gated_inputs(T, D, F, torch.bfloat16, 8)
    h, saved = da.gated_linear_forward(x, wg, wu)
    rows = [0, 1, 65535, 65536, T - 1]
    r = R.gated(x[rows], wg, wu, torch.zeros(5, F, device="cuda"), "silu")
    _close(h[rows], r["h"], R.gated_tolerance(r, torch.bfloat16, "silu")["h"], "h")
    dh = torch.zeros_like(h)
    del h
    dh[-1], dh[0] = 1.0, -1.0
    dx, dg, du = da.gated_linear_backward(dh, x, wg, wu, saved)
    r = R.gated(x[[0, T - 1]], wg, wu, dh[[0, T - 1]], "silu")
    tol = R.gated_tolerance(r, torch.bfloat16, "silu")
    _close(dx[[0, T - 1]], r["dx"], tol["dx"], "dx")
    _close(dg, r["dwg"], tol["dwg"], "dwg")
    _close(du, r["dwu"], tol["dwu"], "dwu")
    assert (dx[1:-1] == 0).all()


# ---------------------------------------------------------------- log probabilities

def _probs_check(x, t, temperature=1.0, top=0, a=None, b=None):
    st = da.new_status()
    r, saved = da.log_probs_forward(x, t, temperature, top, status=st)
    dx = da.log_probs_backward(x, t, saved, a, b, temperature)
    assert da.read_status(st) == 0
    w = R.log_probs(x.reshape(-1, x.shape[-1]), t.reshape(-1), temperature, top, *(None if v is None else v.reshape(-1) for v in (a, b)))
    tol = R.log_probs_tolerance(w, x.dtype, temperature)
    _close(r.log_probs.reshape(-1), w["lp"], tol["lp"], "log_probs")
    _close(r.entropy.reshape(-1), w["H"], tol["H"], "entropy")
    if top:
        assert torch.equal(r.top_indices.reshape(-1, top), w["top"])
        _close(r.top_log_probs.reshape(-1, top), w["top_lp"], tol["lp_all"].gather(1, w["top"]), "top_log_probs")
    if "dx" in w:
        _close(dx.reshape(w["dx"].shape), w["dx"], tol["dx"], "dlogits")
    return r, dx


def _logits(rows, V, dtype, seed=0, by=2.5, gap=0, shift=0):
    g = _gen(seed + rows + V)
    x = _randn(rows, V + gap, g=g, to=dtype, by=by)[:, shift:shift + V]
    t = torch.randint(0, V, (rows,), device="cuda", generator=g)
    return x, t, _randn(rows, g=g), _randn(rows, g=g)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, V, top", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (2, 33, 32), (9, 1000, 20), (4, 2047, 5), (4, 2049, 32), (300, 4099, 1), (1, 8193, 32),
                                          (7, 32003, 7), (1, 128256, 20), (20, 70001, 5), (160, 16385, 20), (700, 9001, 3), (0, 50, 4)])
def test_log_probs(rows, V, top, dtype):
    """Short rows, a CTA a row, clusters of two to eight, vectors that end inside and beyond a step."""
    x, t, a, b = _logits(rows, V, dtype)
    _probs_check(x, t, 1.0, top, a, b)
    _probs_check(x, t, 0.7, 0, a, None)
    _probs_check(x, t, 1.3, min(top, 2), None, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows, V, top", [(1217, 64003, 5), (1300, 128256, 1), (1900, 30001, 7), (2432, 25000, 0), (2500, 64008, 3)])
def test_log_probs_of_more_rows_than_one_round(rows, V, top, dtype):
    """Long rows of which more than one round of CTAs, with two, four and eight warps each."""
    x, t, a, b = _logits(rows, V, dtype)
    _probs_check(x, t, 1.3, top, a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [40, 3001, 40001])
@pytest.mark.parametrize("gap, shift", [(3, 1), (8, 0), (13, 5), (1, 0)])
def test_log_probs_rows_of_wider_buffers(V, gap, shift, dtype):
    x, t, a, b = _logits(6, V, dtype, 1, gap=gap, shift=shift)
    _probs_check(x, t, 1.0, 10, a, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [50, 5000, 100000])
def test_log_probs_masks(V, dtype):
    """-inf in places, in all but one, in all; the type's lowest value in places and in all; targets that are masked or absent."""
    x, t, a, b = _logits(12, V, dtype, 2)
    low = torch.finfo(dtype).min
    x[0, ::3] = -INF
    x[1] = -INF
    x[2] = -INF
    x[2, V // 2] = 1.5
    x[3, : V - 9] = -INF
    x[4, ::2] = low
    x[5] = low
    x[6] = low
    x[6, 7] = -3.0
    x[7] = 0.0
    x[8] = -INF
    x[8, ::V // 4] = low
    t[0], t[1], t[2], t[3], t[4], t[5], t[6], t[7], t[8] = 0, 3, V // 2, 1, 0, 9, 8, 5, 1
    t[9], t[10] = -1, -100
    r, dx = _probs_check(x, t, 1.0, 30, a, b)
    assert r.entropy[1] == 0 and r.log_probs[1] == -INF and (r.top_log_probs[1] == -INF).all() and (dx[1] == 0).all()
    assert r.log_probs[2] == 0 and r.entropy[2] == 0 and (r.log_probs[9:11] == 0).all()
    assert (dx[0, 3::3] == 0).all()                       # -inf has no gradient but as a target
    _probs_check(x, t, 2.0, 5, None, b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [200, 3000, 40000, 128256])
def test_alternatives_of_rows_in_any_order(V, dtype):
    """Growing, falling, constant, few values, one value often, zeros of both signs, the largest at the end."""
    g = _gen(V)
    up = torch.arange(V, device="cuda").float() / V * 8
    two = (torch.arange(V, device="cuda") % 2).float()
    zeros = torch.where(torch.rand(V, device="cuda", generator=g) < 0.5, 0.0, -0.0)
    end = _randn(V, g=g)
    end[-40:] += 20
    x = torch.stack([up, up.flip(0), torch.zeros_like(up), two, (up * 100) % 7, zeros, -up, end, -INF * two.nan_to_num(0).neg().add(1).clamp_min(1e-9)]).to(dtype)
    t = torch.zeros(len(x), dtype=torch.int64, device="cuda")
    for top in (1, 8, 32):
        r = da.log_probs_forward(x, t, 1.0, top)[0]
        want = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(r.top_indices, want), top


def test_log_probs_large_logits_and_temperatures():
    """The difference from the largest is what counts, whatever its size."""
    x, t, a, b = _logits(5, 3000, torch.float32, 4)
    base, saved = da.log_probs_forward(x, t)
    for shift in (2.0 ** 12, -(2.0 ** 12)):                # exact in binary32 up to the grid of the sum
        y = (x * 2048).round() / 2048
        one, two = da.log_probs_forward(y, t, 1.0, 3)[0], da.log_probs_forward(y + shift, t, 1.0, 3)[0]
        for p, q in zip(one, two):
            assert torch.equal(p, q)
    for temperature in (2.0 ** -60, 1e-4, 1e4, 2.0 ** 60):
        _probs_check(x, t, temperature, 5)
    _probs_check(x * 1e18, t, 1e17, 5)


@pytest.mark.parametrize("V", [60, 9000])
def test_log_probs_not_finite(V):
    """NaN or +inf spoils its own row and says so; a target past the last column too."""
    x, t, a, b = _logits(6, V, torch.float32, 5)
    want = da.log_probs_forward(x, t, 1.0, 4)[0]
    x[1, V // 2], x[3, 5] = float("nan"), INF
    st = da.new_status()
    got, saved = da.log_probs_forward(x, t, 1.0, 4, status=st)
    assert da.read_status(st) == da.STATUS_NONFINITE
    dx = da.log_probs_backward(x, t, saved, a, b)
    for row in range(6):
        if row in (1, 3):
            assert got.log_probs[row].isnan() and got.entropy[row].isnan()
            assert ((got.top_indices[row] >= 0) & (got.top_indices[row] < V)).all()
        else:
            assert all(torch.equal(p[row], q[row]) for p, q in zip(got, want)) and torch.isfinite(dx[row]).all()
    x, t, a, b = _logits(6, V, torch.float32, 5)
    t[2], t[4] = V, 2 ** 40
    st.zero_()
    got, saved = da.log_probs_forward(x, t, status=st)
    assert da.read_status(st) == da.STATUS_BAD_TARGET
    assert got.log_probs[[2, 4]].isnan().all() and torch.equal(got.entropy, want.entropy)
    r = R.log_probs(x, t, 1.0, 0, a, b)
    _close(da.log_probs_backward(x, t, saved, a, b), r["dx"], R.log_probs_tolerance(r, torch.float32, 1.0)["dx"], "dlogits")


def test_log_probs_shapes_autograd_and_in_place():
    g = _gen(6)
    x = _randn(3, 4, 500, g=g)
    t = torch.randint(-1, 500, (3, 4), device="cuda", generator=g)
    a, b = _randn(3, 4, g=g), _randn(3, 4, g=g)
    _probs_check(x, t, 1.0, 6, a, b)
    leaf = x.clone().requires_grad_(True)
    r = da.log_probs(leaf, t.int(), 1.0, 6)
    assert r.top_indices.shape == (3, 4, 6)
    ((r.log_probs * a).sum() + (r.entropy * b).sum()).backward()
    want, saved = da.log_probs_forward(x, t)
    dx = da.log_probs_backward(x, t, saved, a, b)
    assert torch.equal(leaf.grad, dx)
    leaf.grad = None
    da.log_probs(leaf, t).entropy.sum().backward()
    assert torch.equal(leaf.grad, da.log_probs_backward(x, t, saved, None, torch.ones_like(b)))
    same = da.log_probs_backward(x, t, saved, a, b, out=x)
    assert same is x and torch.equal(x, dx)
    cols = _randn(500, 12, g=g).T                          # columns that are not contiguous
    _probs_check(cols, t.reshape(-1), 1.0, 6, a.reshape(-1), b.reshape(-1))
    assert da.log_probs_backward(cols, t.reshape(-1), da.log_probs_forward(cols, t.reshape(-1))[1], a.reshape(-1)).shape == cols.shape


def test_log_probs_agree_with_the_exact_cross_entropy():
    """The loss of the exact reduction is minus the log probability; both are within their roundings."""
    x, t, a, _ = _logits(40, 128256, torch.float32, 7)
    loss = da.dce_forward(x, t)[0]
    r, saved = da.log_probs_forward(x, t)
    w = R.log_probs(x, t)
    assert ((loss + r.log_probs).abs() <= R.log_probs_tolerance(w, torch.float32, 1.0)["lp"] + 2.0 ** -23 * loss).all()


def test_log_probs_same_bytes_in_a_graph():
    x, t, a, b = _logits(300, 40000, torch.bfloat16, 8)
    few = x[:5].contiguous()

    def step():
        r, saved = da.log_probs_forward(x, t, 1.0, 5)
        q, _ = da.log_probs_forward(few, t[:5], 1.0, 20)
        return (*r, da.log_probs_backward(x, t, saved, a, b), *q)
    want = [v.clone() for v in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for v in out:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, out))


def test_log_probs_offsets_past_32_bits():
    rows, V = 17000, 128256                                # 2.18e9 logits
    x = torch.zeros(rows, V, device="cuda", dtype=torch.bfloat16)
    x[-1, 77777] = 9.0
    t = torch.full((rows,), 5, device="cuda")
    t[-1] = 77777
    r, saved = da.log_probs_forward(x, t, 1.0, 2)
    w = R.log_probs(x[-2:], t[-2:], 1.0, 2, torch.ones(2, device="cuda"), None)
    tol = R.log_probs_tolerance(w, torch.bfloat16, 1.0)
    _close(r.log_probs[-2:], w["lp"], tol["lp"], "log_probs")
    assert r.top_indices[-1].tolist() == [77777, 0] and r.top_indices[0].tolist() == [0, 1]
    dx = da.log_probs_backward(x, t, saved, torch.ones(rows, device="cuda"))
    _close(dx[-2:], w["dx"], tol["dx"], "dlogits")


# ---------------------------------------------------------------- C ABI

def _matrix(t):
    m = da._Matrix()
    m.ptr, m.rows, m.cols, m.row_stride = t.data_ptr(), t.shape[0], t.shape[1], t.stride(0)
    m.dtype = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[t.dtype]
    return ctypes.byref(m)


def test_outputs_in_wider_buffers():
    """Row strides of the outputs, and what lies between the rows stays as it was."""
    L, t = da.lib(), torch.bfloat16
    x, wg, wu, dh = _gated_inputs(300, 72, 136, t, 10)
    h, saved = da.gated_linear_forward(x, wg, wu)
    want = da.gated_linear_backward(dh, x, wg, wu, saved)
    g = _gen(10)
    ids, dy, w, logits = _words(300, 40, g), _randn(300, 24, g=g), _randn(40, 24, g=g), _randn(300, 40, g=g)
    wide = lambda n, c, to=t: torch.full((n, c + 16), 7.0, device="cuda", dtype=to)  # noqa: E731
    s = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    def check(buffers, wants):
        torch.cuda.synchronize()
        for b, v in zip(buffers, wants):
            c = v.shape[1]
            assert torch.equal(b[:, :c], v) and (b[:, c:] == 7).all()
    for n in (300, 5):
        b = wide(n, 136)
        assert L.dgl_forward(_matrix(x[:n]), _matrix(wg), _matrix(wu), 0, _matrix(b[:, :136]), saved.data_ptr() if n > 5 else None, None, s) == 0
        check([b], [h if n > 5 else da.gated_linear(x[:n], wg, wu)])
    bs = [wide(300, 72), wide(136, 72), wide(136, 72)]
    m = [_matrix(b[:, :72]) for b in bs]
    assert L.dgl_backward(_matrix(dh), _matrix(x), _matrix(wg), _matrix(wu), saved.data_ptr(), *m, ws.data_ptr(), ws.numel(), None, s) == 0
    check(bs, want)
    assert L.dgl_backward(_matrix(dh[:0]), _matrix(x[:0]), _matrix(wg), _matrix(wu), None, None, *m[1:], ws.data_ptr(), ws.numel(), None, s) == 0
    check(bs[1:], [torch.zeros_like(want[1])] * 2)
    f = torch.float32
    bs = [wide(300, 24, f), wide(40, 24, f)]
    assert L.dte_forward(ids.data_ptr(), 64, _matrix(w), 2.0, _matrix(bs[0][:, :24]), None, s) == 0
    assert L.dte_backward(ids.data_ptr(), 64, _matrix(dy), 2.0, -1, _matrix(bs[1][:, :24]), ws.data_ptr(), ws.numel(), None, s) == 0
    check(bs, [da.embedding_forward(ids, w, 2.0), da.embedding_backward(dy, ids, 40, 2.0)])
    for n in (0, 5000):                                    # no tokens; the longer sort
        many, dm, b = _words(n, 40, g), _randn(n, 24, g=g), wide(40, 24, f)
        assert L.dte_backward(many.data_ptr(), 64, _matrix(dm), 1.0, 3, _matrix(b[:, :24]), ws.data_ptr(), ws.numel(), None, s) == 0
        check([b], [da.embedding_backward(dm, many, 40, 1.0, 3)])
    targets, up, b = ids % 40, _randn(300, g=g), wide(300, 40, f)
    _, kept = da.log_probs_forward(logits, targets)
    assert L.dlp_backward(_matrix(logits), targets.data_ptr(), kept.data_ptr(), up.data_ptr(), None, 1.0, _matrix(b[:, :40]), s) == 0
    check([b], [da.log_probs_backward(logits, targets, kept, up)])


# ---------------------------------------------------------------- together

def _decoder_step(p, ids, targets, advantage):
    """Tokens in, log probabilities out: lookup, norm, gated block, norm, logits; a policy-gradient loss with an entropy bonus."""
    x = da.embedding(ids, p["embedding"], 8.0, padding_idx=0)
    h = da.gated_linear(da.layer_norm(x, p["n1"]), p["gate"], p["up"], "silu")
    y = da.layer_norm(x + h @ p["down"].mT, p["n2"])
    r = da.log_probs(y @ p["head"].mT, targets, temperature=0.9)
    return -(r.log_probs * advantage).mean() - 0.01 * r.entropy.mean()


def _decoder_exact(p, ids, targets, advantage):
    p = {k: v.detach().double().requires_grad_(True) for k, v in p.items()}
    emb = torch.where(torch.arange(len(p["embedding"]), device="cuda")[:, None] == 0, p["embedding"].detach(), p["embedding"])
    x = 8.0 * emb[ids]
    n = lambda v, w: torch.nn.functional.layer_norm(v, v.shape[-1:], w)  # noqa: E731
    a = n(x, p["n1"])
    h = torch.nn.functional.silu(a @ p["gate"].mT) * (a @ p["up"].mT)
    z = torch.log_softmax(n(x + h @ p["down"].mT, p["n2"]) @ p["head"].mT / 0.9, -1)
    lp = z.gather(-1, targets.clamp_min(0)[..., None])[..., 0] * (targets >= 0)
    loss = -(lp * advantage.double()).mean() + 0.01 * (z.exp() * z).sum(-1).mean()
    loss.backward()
    return loss.detach(), {k: v.grad for k, v in p.items()}


def test_a_decoder_step():
    """The operators in a row: the loss and every gradient against 64 bits, the same bytes twice, and an AdamW step of them.
    A gradient passes some ten roundings of 2^-9 of its mean size at most: 10 x 2^-9 of its norm is allowed."""
    g = _gen(9)
    t = torch.bfloat16
    p = {"embedding": _randn(700, 256, g=g, to=t, by=0.1), "n1": torch.ones(256, device="cuda"), "gate": _randn(512, 256, g=g, to=t, by=1 / 16),
         "up": _randn(512, 256, g=g, to=t, by=1 / 16), "down": _randn(256, 512, g=g, to=t, by=0.05), "n2": torch.ones(256, device="cuda"),
         "head": _randn(700, 256, g=g, to=t, by=1 / 16)}
    ids, targets = torch.randint(0, 700, (4, 90), device="cuda", generator=g), torch.randint(-1, 700, (4, 90), device="cuda", generator=g)
    ids[:, -3:] = 0
    advantage = _randn(4, 90, g=g)
    runs = []
    for _ in range(2):
        q = {k: v.clone().requires_grad_(True) for k, v in p.items()}
        loss = _decoder_step(q, ids, targets, advantage)
        loss.backward()
        grads = {k: v.grad.clone() for k, v in q.items()}
        opt = da.AdamW(list(q.values()), lr=1e-2)
        opt.step()
        runs.append((loss.detach(), grads, q))
    exact, want = _decoder_exact(p, ids, targets, advantage)
    assert abs(runs[0][0].double() - exact) <= 10 * 2.0 ** -9 * (1 + exact.abs())
    for k in p:
        off = (runs[0][1][k].double() - want[k]).norm() / want[k].norm()
        assert off <= 10 * 2.0 ** -9, (k, float(off))
        assert torch.equal(runs[0][1][k], runs[1][1][k]) and torch.equal(runs[0][2][k], runs[1][2][k])
    assert (runs[0][1]["embedding"][0] == 0).all() and math.isfinite(float(exact))
