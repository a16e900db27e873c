"""Launch plans of window attention that need longer lists or other shapes than
test_gpu_window's: clusters that share a query tile of dq, among them."""
import pytest
import torch

from block_sparse_full_b200 import ssa
from test_gpu_window import _dev, _make, _run

pytestmark = pytest.mark.gpu

# B, Hq, Hkv, T, D, window, sinks, lens: 32 key tiles of 64 and more to a query tile
SHARED = [
    (1, 1, 1, 2500, 128, 0, 0, None),
    (1, 2, 1, 2600, 64, 2100, 100, None),        # sinks' tiles among the stretches
    (1, 2, 2, 3001, 128, 2050, 17, None),
    (2, 1, 1, 2304, 128, 0, 0, [2304, 600]),     # ranks without a tile
    (2, 2, 1, 2600, 64, 2070, 128, [2500, 513]),
    (2, 1, 1, 2400, 128, 2300, 3, [0, 2400]),
]


@pytest.mark.parametrize("case", SHARED, ids=str)
def test_shared_query_tiles(case):
    B, Hq, Hkv, T, D, window, sinks, lens = case
    _run(B, Hq, Hkv, T, D, "bf16", window, sinks, lens=lens, rows=B > 1, seed=T)


def test_shared_query_tiles_on_two_streams():
    # two calls in flight, and one captured and replayed: bit for bit the same
    def make(seed):
        q, k, v, dh = map(_dev, _make(1, 2, 1, 2600, 64, "bf16", False, seed))
        return ssa.window_params_for(q, k, 2100, 100), q, k, v, dh

    def both(c):
        p, q, k, v, dh = c
        out = ssa.window_fwd(p, q, k, v)
        return (out["h"], out["lse"]) + tuple(ssa.window_bwd(p, q, k, v, out, dh))

    calls = [make(1), make(2)]
    want = [both(c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(both(calls[i]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = both(calls[0])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    got[0].append(held)
    ssa.device_status()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(x, y) for x, y in zip(w, r))
