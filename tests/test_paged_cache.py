"""What PagedCache refuses (no GPU needed)."""
import pytest
import torch

from block_sparse_full_b200 import ssa


def _cache(**kw):
    a = {**dict(B=2, Hq=4, Hkv=2, D=64, capacity=100, dtype=torch.bfloat16, device="cpu", page=16), **kw}
    return ssa.PagedCache(**a)


def test_window_behind_a_prefix_is_refused_when_the_cache_is_made():
    # ssa_prefix_decode has no window: the cache could be filled and never read
    with pytest.raises(ssa.SsaError, match="window"):
        _cache(window=5, prefix_len=40)
    p = _cache(prefix_len=40).params
    p.window = 5
    assert ssa.ssa_cache_workspace_size(p, 40) == ssa.ctypes.c_size_t(-1).value and "window" in ssa.ssa_last_error()
    assert 0 < ssa.ssa_cache_workspace_size(p, 0) < 1 << 30
    assert _cache(window=5).params.window == 5


def test_fill_prefix_takes_the_whole_prefix():
    # fewer tokens would leave rows of zeros that attend() weighs as tokens
    c = _cache(prefix_len=40)
    rows = lambda n: torch.ones(n, 2, 64, dtype=torch.bfloat16)  # noqa: E731
    for n in (39, 41, 48, 0):
        with pytest.raises(ValueError, match="40"):
            c.fill_prefix(rows(n), rows(n))
    with pytest.raises(ValueError, match="40"):
        c.fill_prefix(rows(40), rows(39))
    with pytest.raises(ValueError, match="CUDA"):  # the right number of tokens reaches the call itself
        c.fill_prefix(rows(40), rows(40))
    with pytest.raises(ValueError, match="no shared prefix"):
        _cache().fill_prefix(rows(40), rows(40))
