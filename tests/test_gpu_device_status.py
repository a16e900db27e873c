"""One status call reports the gravest record of the work before it and clears all of them."""
import pytest
import torch

from block_sparse_full_b200 import ssa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _status():
    return ssa.ssa_device_status(torch.cuda.current_stream().cuda_stream)


def _window(dtype, lens):
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, dh = (torch.randn(2, 2, 100, 64, generator=g, device=DEV).to(DT[dtype]) for _ in range(4))
    p = ssa.window_params_for(q, k, 10, 0)
    lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    f = ssa.window_fwd(p, q, k, v, lens=lens)
    ssa.window_bwd(p, q, k, v, f, dh, lens=lens)


def _step(dtype, last_page):
    g = torch.Generator(device=DEV).manual_seed(2)
    pool = torch.zeros(4, 1, 16, 64, device=DEV).to(DT[dtype])
    table = torch.tensor([[0, 1], [2, last_page]], dtype=torch.int32, device=DEV)
    x = torch.randn(2, 1, 64, generator=g, device=DEV).to(DT[dtype])
    p = ssa.cache_params_for(x, pool, table)
    lens = torch.tensor([30, 16], dtype=torch.int32, device=DEV)
    lens = ssa.cache_append(p, pool, pool.clone(), table, lens, x, x, q=x)["lens"]
    ssa.paged_decode(p, x, pool, pool, table, lens)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_length_in_two_kernels_is_reported_once(dtype):
    assert _status() == ssa.SSA_OK
    _window(dtype, [101, 50])
    assert _status() == ssa.SSA_ERR_INVALID_ARG and "length" in ssa.ssa_last_error()
    _window(dtype, [100, 50])
    assert _status() == ssa.SSA_OK and not ssa.ssa_last_error()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_page_in_two_kernels_is_reported_once(dtype):
    assert _status() == ssa.SSA_OK
    _step(dtype, 9)
    assert _status() == ssa.SSA_ERR_INVALID_ARG and "out of range" in ssa.ssa_last_error()
    _step(dtype, 3)
    assert _status() == ssa.SSA_OK


def test_an_expired_wait_is_graver_than_an_argument():
    assert _status() == ssa.SSA_OK
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    for dtype in ("bf16", "f32"):
        _window(dtype, [-1, 101])
        _step(dtype, -2)
    stream = torch.cuda.current_stream().cuda_stream
    assert ssa.ssa_selftest_wait_timeout(1_000_000, flag.data_ptr(), stream) == ssa.SSA_OK
    assert _status() == ssa.SSA_ERR_TIMEOUT and "expired" in ssa.ssa_last_error()
    assert _status() == ssa.SSA_OK and not ssa.ssa_last_error()
