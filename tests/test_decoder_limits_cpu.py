"""Host-side checks of the decoder's operators: outputs that share memory with inputs."""
import os
import random
import sys

import pytest
import torch

import bitwise_deterministic_shard_gb300 as da
from bitwise_deterministic_shard_gb300 import decoder, train

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_decoder_cpu import stub  # noqa: E402,F401


def test_outputs_may_not_share_memory_with_inputs(stub):  # noqa: F811
    """An output on an input, or on a part of one, is refused before the library; beside it, or between its rows, it is taken."""
    t = torch.bfloat16
    x, w, v = torch.zeros(16, 16, dtype=t), torch.zeros(16, 16, dtype=t), torch.zeros(16, 16, dtype=t)
    for out in (x, w, v):
        with pytest.raises(da.DetAttnError, match="share memory"):
            da.gated_linear_forward(x, w, v, out=out)
    buffer = torch.zeros(800, dtype=t)
    x = buffer[256:512].view(16, 16)
    for start, taken in ((0, True), (8, False), (256, False), (504, False), (512, True)):
        out = buffer[start:start + 256].view(16, 16)
        if taken:
            assert da.gated_linear_forward(x, w, v, out=out)[0] is out
        else:
            with pytest.raises(da.DetAttnError, match="share memory"):
                da.gated_linear_forward(x, w, v, out=out)
    rows = torch.zeros(4, 320, dtype=t)                    # 16 columns of a wider buffer: the other 304 of a row are free
    for start, taken in ((16, True), (320 + 64, True), (8, False), (3 * 320 + 16, True), (896, True), (904, False)):
        out = rows.view(-1)[start:start + 64].view(4, 16)
        if taken:
            da.gated_linear_forward(rows[:, :16], w, v, out=out)
        else:
            with pytest.raises(da.DetAttnError, match="share memory"):
                da.gated_linear_forward(rows[:, :16], w, v, out=out)
    x = torch.zeros(16, 32, dtype=t)[:, ::2]               # copied before it is read, so its memory is free
    da.gated_linear_forward(x, w, v, out=x._base.view(-1)[:256].view(16, 16))
    da.gated_linear_forward(x[:0], w, v, out=w[:0])        # nothing is written

    e = torch.zeros(10, 8)
    ids = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(da.DetAttnError, match="share memory"):
        da.embedding_forward(ids, e, out=e[2:5])
    da.embedding_forward(ids, e[:2], out=e[2:5])


def test_a_gradient_may_lie_on_its_logits(stub):  # noqa: F811
    buffer = torch.zeros(100)
    z, n, g = buffer[:36].view(4, 9), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    _, saved = da.log_probs_forward(z, n)
    for out, taken in ((z, True), (buffer[36:72].view(4, 9), True), (buffer[4:40].view(4, 9), False), (buffer[35:71].view(4, 9), False)):
        if taken:
            assert da.log_probs_backward(z, n, saved, g, out=out) is out
        else:
            with pytest.raises(da.DetAttnError, match="share memory"):
                da.log_probs_backward(z, n, saved, g, out=out)
    wide = torch.zeros(4, 12)[:, :9]                       # the logits' start, but other rows
    with pytest.raises(da.DetAttnError, match="share memory"):
        da.log_probs_backward(wide, n, saved, g, out=wide._base.view(-1)[:36].view(4, 9))
    one = buffer[:9].view(1, 9)
    assert da.log_probs_backward(one, n[:1], saved[:1], g[:1], out=one) is one


def test_shared_memory_against_sets_of_places():
    g = random.Random(0)
    buffer = torch.zeros(200, dtype=torch.int16)
    for _ in range(20000):
        rows, cols, at, n, o = g.randint(0, 5), g.randint(1, 9), g.randint(0, 50), g.randint(1, 30), g.randint(0, 120)
        run = cols + g.randint(0, 15)
        shared = {at + i * run + c for i in range(rows) for c in range(cols)} & set(range(o, o + n))
        try:
            decoder._apart(buffer[o:o + n], train._MATRIX.pack(buffer.data_ptr() + 2 * at, 1, rows, cols, run))
            refused = False
        except da.DetAttnError:
            refused = True
        assert refused == bool(shared)
