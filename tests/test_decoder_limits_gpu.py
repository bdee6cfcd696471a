"""The decoder's operators at their limits: results of a few bytes, logits as far apart as their type allows, factors beside a
rounding, rows of which little is finite, and two calls at once on new inputs."""
import ctypes
import os
import sys

import pytest
import torch

import bitwise_deterministic_shard_gb300 as da

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
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
