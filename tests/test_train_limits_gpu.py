"""The training operators at the ends of their ranges: scores of any size, caps of any size, padding that fills whole
warps, values that may not matter, infinite gradients, gradients that come late."""
import os
import sys

import numpy as np
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
