"""Rows of window attention whose query is not a finite number."""
import math

import pytest
import torch

from block_sparse_full_b200 import ssa
from test_gpu_window import _dev, _make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 2, 1, 130, 64, 0, 0), (1, 1, 1, 1500, 128, 300, 4), (2, 16, 4, 700, 128, 100, 3)],
                         ids=str)
def test_query_of_nan(shape, dtype):
    # outside the contract (rows before a length are finite), yet it stays in its row and is not taken for an empty one
    B, Hq, Hkv, T, D, window, sinks = shape
    q, k, v, _ = map(_dev, _make(B, Hq, Hkv, T, D, dtype, seed=4))
    p = ssa.window_params_for(q, k, window, sinks)
    want = ssa.window_fwd(p, q, k, v)
    rows = torch.zeros(B, Hq, T, dtype=torch.bool, device=q.device)
    rows[0, 0, 0] = rows[-1, -1, T - 1] = rows[0, Hq // 2, T // 2] = True
    q[rows] = math.nan
    got = ssa.window_fwd(p, q, k, v)
    torch.cuda.synchronize()
    ssa.device_status()
    assert torch.isnan(got["h"][rows]).all() and torch.isnan(got["lse"][rows]).all()
    assert torch.equal(got["h"][~rows], want["h"][~rows]) and torch.equal(got["lse"][~rows], want["lse"][~rows])
