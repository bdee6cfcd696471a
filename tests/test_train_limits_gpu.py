"""The training operators at the ends of their ranges: scores of any size, caps of any size, padding that fills whole
warps, values that may not matter, infinite gradients, gradients that come late."""
import os
import sys

import pytest
import torch

import bitwise_deterministic_shard_gb300 as da

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import test_train_gpu as T  # noqa: E402
import train_reference as R  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


# ---------------------------------------------------------------- padding

@pytest.mark.parametrize("pad_id", [-1, -9])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B, H", [(1, 4), (6, 16)])      # groups of a CTA that share a query tile; a tile each
@pytest.mark.parametrize("S, pad", [(256, 32), (256, 64), (256, 96), (512, 32), (512, 160), (300, 44)])
def test_padding_that_fills_whole_warps(S, pad, B, H, causal, pad_id):
    """The last queries are padding in runs of 32, the rows of a warp; all others are one document."""
    q, k, v, go = T._attn_inputs(B, H, H // 2, S, S, 64, torch.bfloat16, seed=S + pad)
    docs = torch.full((B, S), 7, dtype=torch.int32, device="cuda")
    docs[:, S - pad:] = pad_id
    out, lse, dq, dk, dv = T._attn_check(q, k, v, go, causal=causal, docs=docs)
    assert (out[:, :, S - pad:] == 0).all() and (lse[:, :, S - pad:] == -float("inf")).all()
    q[:, :, S - pad:] = float("nan")
    st = da.new_status()
    again = da.attention_forward(q, k, v, causal=causal, docs=docs, status=st)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse) and da.read_status(st) == 0


# ---------------------------------------------------------------- scores of any size

def _tall(B, Hq, Hkv, Sq, Skv, dtype, base, late):
    """Products that are exact in binary32: 16 dimensions give every score +-256 |base| times a power of two (scale 1/4),
    the others a spread of about 3.5.  late: the first half of the keys without the common part."""
    g = torch.Generator(device="cuda").manual_seed(int(abs(base) * 2) + Skv)
    q = torch.randint(-2, 3, (B, Hq, Sq, 64), device="cuda", generator=g).to(dtype)
    k = torch.randint(-2, 3, (B, Hkv, Skv, 64), device="cuda", generator=g).to(dtype)
    q[..., :16], k[..., :16] = 64, base
    if late:
        k[:, :, :Skv // 2, :16] = 0
    v, go = (torch.randn(B, h, s, 64, device="cuda", generator=g).to(dtype) for h, s in ((Hkv, Skv), (Hq, Sq)))
    return q, k, v, go


TALL = [(1, 2, 1, 150, 300), (5, 16, 16, 130, 260), (2, 8, 2, 1, 1500), (1, 4, 4, 1, 70)]


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("base", [5.0, 11.5, -11.5, 23.5, -23.5, 60.0, -60.0, 156.0, -156.0])   # scores of 1280 to 39936
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", TALL)
def test_tall_scores(shape, dtype, base, late):
    """The output's roundings do not depend on the size of the scores; lse is one binary32 number, so the weights that the
    backward pass forms from it are off by six roundings of it, a factor of a row."""
    q, k, v, go = _tall(*shape, dtype, base, late)
    kw = dict(causal=True, scale=0.25)
    st = da.new_status()
    out, lse = da.attention_forward(q, k, v, status=st, **kw)
    r = R.attention(q, k, v, go, **kw)
    tol, A = R.attention_tolerance(r, dtype), r["abs"]
    T._close(out, r["out"], tol["out"], "out")
    assert ((lse.double() - r["lse"]).abs() <= 2.0 ** -17 * (1 + r["lse"].abs())).all()
    grads = da.attention_backward(q, k, v, out, lse, go, status=st, **kw)
    e = 6 * 2.0 ** -24 * float(r["lse"].abs().max())
    for got, n, more in zip(grads, ("dq", "dk", "dv"), (2 * A["dq_rough"], 2 * A["dk_rough"], A["dv"])):
        T._close(got, r[n], tol[n] + e * more, n)
    assert da.read_status(st) == 0


# ---------------------------------------------------------------- caps of any size

@pytest.mark.parametrize("shape", [(1, 4, 2, 200, 300, 64), (6, 16, 16, 130, 260, 64), (2, 8, 2, 1, 1500, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("cap", [1e-3, 0.1, 31.0, 32.0, 33.0, 50.0, 300.0, 400.0, 1e4, 1e5, 1e6, 1e9])
def test_caps(shape, dtype, cap):
    """The capped score is off by 2^-21 of the cap where it is a good part of the cap, and by 2^-22 of itself below a quarter
    of a cap beyond 4096 times the scale, where every score here lies."""
    q, k, v, go = T._attn_inputs(*shape, dtype, seed=12)
    kw = dict(causal=True, softcap=cap)
    st = da.new_status()
    out, lse = da.attention_forward(q, k, v, status=st, **kw)
    dq, dk, dv = da.attention_backward(q, k, v, out, lse, go, status=st, **kw)
    assert da.read_status(st) == 0
    r = R.attention(q, k, v, go, **kw)
    tol, A = R.attention_tolerance(r, dtype), r["abs"]
    e = min(cap, 362.0) * 2.0 ** -21
    for got, n, more in ((out, "out", 2 * A["out"]), (dq, "dq", 4 * A["dq_rough"]), (dk, "dk", 4 * A["dk_rough"]), (dv, "dv", 2 * A["dv"])):
        T._close(got, r[n], tol[n] + e * more, n)
    assert ((lse.double() - r["lse"]).abs() <= 2.0 ** -17 * (1 + r["lse"].abs()) + e).all()


def test_a_large_cap_is_no_cap():
    """u = t - t^3 / (3 cap^2): at 1e6 the scores of up to 2^6 are the products to 2^-24 of them, so lse is the one without a
    cap up to the roundings of both."""
    q, k, v, _ = T._attn_inputs(2, 4, 2, 200, 300, 64, torch.bfloat16, seed=13)
    want = da.attention_forward(q, k, v)[1]
    for cap in (1e6, 1e9, 1e15):
        lse = da.attention_forward(q, k, v, softcap=cap)[1]
        assert ((lse - want).abs() <= 2.0 ** -18 * (1 + want.abs())).all(), cap


@pytest.mark.parametrize("cap", [1e-8, 1e-12])
def test_scores_of_zero_under_a_tiny_cap(cap):
    """Without a score other than 0 every key weighs the same."""
    q = torch.zeros(1, 2, 200, 64, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn(1, 2, 200, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    T._attn_check(q, k, v, torch.randn_like(q), softcap=cap)


# ---------------------------------------------------------------- what may not matter

def _leave_behind(x):
    """Fills the shared memory of every SM where a query tile lies: a call whose output is x everywhere."""
    q = torch.full((4, 152, 256, 128), x, device="cuda", dtype=torch.bfloat16)
    da.attention_forward(q, q, q, scale=0.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B, Hkv, group, Sq, Skv", [(2, 2, 5, 24, 200), (2, 1, 3, 40, 1200), (1, 2, 7, 18, 90), (90, 2, 5, 25, 130)])
def test_rows_that_are_no_query(B, Hkv, group, Sq, Skv, dtype):
    """Heads that do not divide 128 leave rows of the query tile unfilled: what lies there decides nothing."""
    q, k, v, _ = T._attn_inputs(B, Hkv * group, Hkv, Sq, Skv, 128, dtype, seed=14, heavy=False)
    kw = dict(causal=True, softcap=30.0)
    _leave_behind(0.0)
    want = da.attention_forward(q, k, v, **kw)
    for x in (300.0, 10.0, 3.0, 1.5, 0.7):
        for _ in range(4):
            _leave_behind(x)
            got = da.attention_forward(q, k, v, **kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), x


@pytest.mark.parametrize("B, H, Sq", [(1, 4, 320), (6, 16, 320), (2, 8, 1)])
def test_padding_does_not_matter(B, H, Sq):
    """Tokens of padding, of any size: the same bytes, whichever form of the cap their scores would take."""
    S = 320
    q, k, v, go = T._attn_inputs(B, H, H // 2, Sq, S, 64, torch.bfloat16, seed=15, heavy=False)
    docs = torch.zeros(B, S, dtype=torch.int32, device="cuda")
    docs[:, 100:110] = -1
    kw = dict(causal=True, softcap=30.0, docs=docs)

    def both(q, k):
        out, lse = da.attention_forward(q, k, v, **kw)
        return out, lse, *da.attention_backward(q, k, v, out, lse, go, **kw)
    want = both(q, k)
    for x in (2.0, 8.0, 300.0, 1e30, float("nan")):
        kk, qq = k.clone(), q.clone()
        kk[:, :, 100:110] *= x
        if Sq == S:
            qq[:, :, 100:110] *= x
        for a, b in zip(both(qq, kk), want):
            assert torch.equal(a, b), x


# ---------------------------------------------------------------- layer norm

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_layer_norm_bias_keeps_its_type(dtype):
    """An f32 bias beside 16-bit rows without a weight: its gradient is a binary32 sum, not a 16-bit one."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(700, 300, device="cuda", generator=g).to(dtype)
    dy = (torch.randn(700, 300, device="cuda", generator=g) + 200).to(dtype)     # sums of 140000, beyond f16
    b = torch.zeros(300, device="cuda", requires_grad=True)
    da.layer_norm(x, None, b).backward(dy)
    r = R.layer_norm(x, None, b.detach(), dy)
    T._close(b.grad, r["db"], R.layer_norm_tolerance(r, dtype, torch.float32, 700, 300)["db"], "db")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows, cols, gap", [(1300, 1100, 0), (400, 1101, 3), (300, 600, 0), (5, 9000, 7)])
def test_layer_norm_bytes_with_the_same_alignment(rows, cols, gap, dtype):
    """Equal values whose rows start alike relative to 16 bytes give equal bytes, wherever they lie."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = (torch.randn(rows, cols, device="cuda", generator=g).to(dtype) for _ in range(2))
    w, b = (torch.randn(cols, device="cuda", generator=g) for _ in range(2))

    def both(x, dy):
        y, mean, rstd = da.layer_norm_forward(x, w, b)
        return y, mean, rstd, *da.layer_norm_backward(dy, x, w, mean, rstd)

    def placed(t, pad):
        room = torch.empty(pad + rows * (cols + gap), device="cuda", dtype=dtype)
        p = room[pad:].view(rows, cols + gap)[:, :cols]
        return p.copy_(t)
    want = both(placed(x, 0), placed(dy, 0))
    for pad in (64, 4096):
        for p, q in zip(both(placed(x, pad), placed(dy, pad)), want):
            assert torch.equal(p, q)


# ---------------------------------------------------------------- AdamW

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan"), 1e25])
def test_adamw_8bit_keeps_an_infinity_to_itself(bad, dtype):
    """A gradient that is not finite, or whose square is not, spoils its own element of an 8-bit block and no other."""
    g = torch.Generator().manual_seed(3)
    ps = [torch.randn(1000, generator=g).to(dtype).cuda() for _ in range(2)]
    ps[1].copy_(ps[0])
    opts = [da.AdamW([p], state_bits=8, **T.H) for p in ps]
    for step in range(3):
        gr = torch.randn(1000, generator=g).to(dtype).cuda()
        for p, x in zip(ps, (0.0, bad)):
            p.grad = gr.clone()
            p.grad[300] = x if step == 0 else 0.0
        for o in opts:
            o.step()
    rest = torch.arange(1000, device="cuda") != 300
    assert torch.isfinite(ps[1][rest]).all()
    if bad == 1e25:                  # a finite first moment, under whose scale the block's others become zero
        return
    assert torch.equal(ps[0][rest], ps[1][rest])
    a, b = (o.groups[0] for o in opts)
    rest = torch.arange(1024, device="cuda") != 300
    for n in ("exp_avg", "exp_avg_sq"):
        assert torch.equal(a[n].view(torch.uint8)[rest], b[n].view(torch.uint8)[rest])
    for n in ("exp_avg_scale", "exp_avg_sq_scale"):
        assert torch.equal(a[n], b[n])


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_first_gradient_that_comes_late(bits):
    """A parameter's bias correction counts its own steps: with a first gradient in the third step it moves as one whose
    first step this is."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(500, generator=g).cuda()
    a, late, fresh = x.clone(), x.clone(), x.clone()
    opt, other = da.AdamW([a, late], state_bits=bits, **T.H), da.AdamW([fresh], state_bits=bits, **T.H)
    for step in range(5):
        gr = torch.randn(500, generator=g).cuda()
        a.grad = gr
        late.grad = gr if step >= 2 else None
        opt.step()
        if step >= 2:
            fresh.grad = gr
            other.step()
    assert torch.equal(late, fresh) and not torch.equal(a, late)
