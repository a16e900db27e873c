"""The waits of the window and prefix kernels run out, kernel by kernel: the call
ends and is reported, and later calls are bit for bit what they were.  With the
wait limit at 1 ns the barrier of the first scores expects one arrival more than
it gets, so the wait for it cannot succeed; nothing faults, and every wait that
follows gives up in turn."""
import pytest
import torch

from block_sparse_full_b200 import ssa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _status():
    return ssa.ssa_device_status(torch.cuda.current_stream().cuda_stream)


def _expires(call, kernels):
    """call() under the limit of 1 ns: reported once, by these kernels and no others."""
    assert _status() == ssa.SSA_OK
    ssa.ssa_debug_set_wait_limit_ns(1)
    try:
        call()
        assert _status() == ssa.SSA_ERR_TIMEOUT
        error = ssa.ssa_last_error()
        assert _status() == ssa.SSA_OK
    finally:
        ssa.ssa_debug_set_wait_limit_ns(0)
    for name in ("attn_tc_kernel", "window_dq_kernel", "window_dkdv_kernel"):
        assert (name in error) == (name in kernels), error


def _same(call, want):
    got = call()
    assert _status() == ssa.SSA_OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))


# B, Hq, Hkv, T, D, window, sinks: one CTA to a tile and clusters, with and without delta's sweep, sinks out of reach
SHAPES = [
    (2, 4, 2, 300, 64, 0, 0),
    (1, 1, 1, 1, 128, 0, 0),
    (4, 16, 4, 1300, 128, 100, 5),
    (4, 16, 4, 1300, 64, 600, 70),
    (1, 1, 1, 2500, 128, 0, 0),
    (1, 2, 1, 2600, 64, 2100, 100),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_window(shape):
    B, Hq, Hkv, T, D, window, sinks = shape
    g = torch.Generator(device=DEV).manual_seed(T)
    q, k, v, dh = (torch.randn(B, H, T, D, generator=g, device=DEV).bfloat16() for H in (Hq, Hkv, Hkv, Hq))
    p = ssa.window_params_for(q, k, window, sinks)
    fwd = ssa.window_fwd(p, q, k, v)
    forward = lambda: list(ssa.window_fwd(p, q, k, v).values())  # noqa: E731
    backward = lambda: list(ssa.window_bwd(p, q, k, v, fwd, dh))  # noqa: E731
    want = forward(), backward()
    _expires(forward, ["attn_tc_kernel"])
    _same(forward, want[0])
    _expires(backward, ["window_dq_kernel", "window_dkdv_kernel"])
    _same(backward, want[1])


@pytest.mark.parametrize("D,page,prefix", [(128, 64, 500), (64, 16, 3000)])
def test_prefix(D, page, prefix):
    g = torch.Generator(device=DEV).manual_seed(D)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    c = ssa.PagedCache(20, 4, 2, D, 64, torch.bfloat16, DEV, page=page, prefix_len=prefix)
    c.fill_prefix(rnd(prefix, 2, D), rnd(prefix, 2, D))
    c.append(rnd(100, 2, D), rnd(100, 2, D))
    x = rnd(20, 4, D)
    call = lambda: list(c.attend(x).values())  # noqa: E731
    want = call()
    _expires(call, ["attn_tc_kernel"])
    _same(call, want)
