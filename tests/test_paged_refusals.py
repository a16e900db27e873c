"""Arguments that window attention and the paged cache refuse, before anything
is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from block_sparse_full_b200 import ssa

A = 1 << 20  # an aligned address that is never read
BAD = ctypes.c_size_t(-1).value


def view(data=A, b=1 << 16, h=1 << 12, t=128):
    return ssa.ssa_view_t(data, b, h, t)


def wp(**kw):
    a = {**dict(B=2, Hq=4, Hkv=2, T=100, D=128, window=16, sinks=4, dtype=ssa.SSA_BF16), **kw}
    return ssa.window_params(a["B"], a["Hq"], a["Hkv"], a["T"], a["D"], a["window"], a["sinks"], a["dtype"],
                             a.get("sm_scale"), a.get("flags", 0))


def cp(**kw):
    a = {**dict(B=2, Hq=4, Hkv=2, D=128, page=64, n_pages=8, max_pages=4, dtype=ssa.SSA_BF16), **kw}
    return ssa.cache_params(**a)


HEADS = [
    (dict(B=0), ssa.SSA_ERR_INVALID_ARG),
    (dict(Hq=3), ssa.SSA_ERR_INVALID_ARG),
    (dict(Hkv=0), ssa.SSA_ERR_INVALID_ARG),
    (dict(D=96), ssa.SSA_ERR_UNSUPPORTED),
    (dict(window=-1), ssa.SSA_ERR_INVALID_ARG),
    (dict(sinks=-1), ssa.SSA_ERR_INVALID_ARG),
    (dict(sinks=129), ssa.SSA_ERR_UNSUPPORTED),
    (dict(dtype=5), ssa.SSA_ERR_INVALID_ARG),
    (dict(sm_scale=0.0), ssa.SSA_ERR_INVALID_ARG),
    (dict(sm_scale=float("nan")), ssa.SSA_ERR_INVALID_ARG),
    (dict(B=70000), ssa.SSA_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", HEADS + [
    (dict(T=0), ssa.SSA_ERR_INVALID_ARG),
    (dict(T=(1 << 30) + 1), ssa.SSA_ERR_UNSUPPORTED),
    (dict(flags=1), ssa.SSA_ERR_INVALID_ARG),
])
def test_window_params(kw, code):
    p, v = wp(**kw), view()
    assert ssa.ssa_window_fwd(p, v, v, v, None, v, A, None) == code, ssa.ssa_last_error()
    assert ssa.ssa_last_error()
    assert ssa.ssa_window_bwd(p, v, v, v, None, v, A, v, v, v, v, A, 1 << 40, None) == code
    assert ssa.ssa_window_workspace_size(p) == BAD


@pytest.mark.parametrize("bad,what", [
    (None, "NULL"), (view(None), "NULL"), (view(A + 2), "aligned"), (view(t=64), "token stride"),
    (view(h=0), "head stride"), (view(b=-128), "batch stride"), (view(t=132), "16 bytes"),
])
def test_window_views(bad, what):
    p, v = wp(), view()
    for i in range(4):
        a = [v, v, v, v]
        a[i] = bad
        assert ssa.ssa_window_fwd(p, *a[:3], None, a[3], A, None) == ssa.SSA_ERR_INVALID_ARG
        assert what in ssa.ssa_last_error()
    for i in range(8):
        a = [v] * 8
        a[i] = bad
        st = ssa.ssa_window_bwd(p, *a[:3], None, a[3], A, *a[4:], A, 1 << 40, None)
        assert st == ssa.SSA_ERR_INVALID_ARG and what in ssa.ssa_last_error()


def test_window_workspace():
    p, v = wp(), view()
    n = ssa.ssa_window_workspace_size(p)
    assert 0 < n < 1 << 30
    assert ssa.ssa_window_bwd(p, v, v, v, None, v, A, v, v, v, v, A, n - 1, None) == ssa.SSA_ERR_WORKSPACE
    assert ssa.ssa_window_bwd(p, v, v, v, None, v, A, v, v, v, v, None, n, None) == ssa.SSA_ERR_WORKSPACE
    assert ssa.ssa_window_bwd(p, v, v, v, None, v, A, v, v, v, v, A + 16, n, None) == ssa.SSA_ERR_INVALID_ARG


def append(p, n=4, k=view(), v=view(), q=None, kp=A, vp=A, table=A, lens=A, new=None, start=None, f=A, rot=64, inter=0,
           off=0, qo=None, ko=None):
    return ssa.ssa_cache_append(p, n, k, v, q, kp, vp, table, lens, new, start, f, rot, inter, off, qo, ko, None)


CACHE = HEADS + [
    (dict(page=8), ssa.SSA_ERR_UNSUPPORTED),
    (dict(page=48), ssa.SSA_ERR_UNSUPPORTED),
    (dict(n_pages=0), ssa.SSA_ERR_INVALID_ARG),
    (dict(max_pages=0), ssa.SSA_ERR_INVALID_ARG),
    (dict(max_pages=1 << 26), ssa.SSA_ERR_UNSUPPORTED),
    (dict(page_stride=100), ssa.SSA_ERR_INVALID_ARG),
    (dict(page_stride=2 * 64 * 128 + 4), ssa.SSA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,code", CACHE)
def test_cache_params(kw, code):
    p, v = cp(**kw), view()
    assert append(p) == code, ssa.ssa_last_error()
    assert ssa.ssa_paged_decode(p, v, A, A, A, A, v, A, A, 1 << 40, None) == code
    assert ssa.ssa_prefix_decode(p, v, A, A, A, 10, A, A, v, A, A, 1 << 40, None) == code
    assert ssa.ssa_cache_workspace_size(p, 0) == BAD


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(n=3), dict(rot=63), dict(rot=130), dict(rot=-2), dict(off=-1), dict(f=None), dict(q=view()),
    dict(qo=view()), dict(k=None), dict(v=view(None)), dict(kp=None), dict(vp=A + 4), dict(table=None), dict(lens=None),
    dict(new=A + 16, lens=A + 20), dict(k=view(t=0)), dict(ko=view(h=4)), dict(start=A + 2),
    dict(f=A + 4), dict(lens=A + 1),
])
def test_append_arguments(kw):
    p = cp(B=2) if "new" not in kw else cp(B=100)
    if "new" in kw:
        kw = {**kw, "n": 100, "lens": A, "new": A + 16}
    assert append(p, **kw) == ssa.SSA_ERR_INVALID_ARG
    assert ssa.ssa_last_error()


def test_decode_arguments():
    p, v = cp(), view()
    n = ssa.ssa_cache_workspace_size(p, 0)
    m = ssa.ssa_cache_workspace_size(p, 1000)
    assert 0 < n < m

    def dec(q=v, kp=A, vp=A, t=A, lens=A, h=v, lse=A, ws=A, nb=n):
        return ssa.ssa_paged_decode(p, q, kp, vp, t, lens, h, lse, ws, nb, None)

    for kw in (dict(lens=A + 2), dict(lse=A + 1), dict(t=A + 3), dict(q=None), dict(kp=None), dict(vp=None), dict(t=None), dict(lens=None), dict(h=None), dict(lse=None),
               dict(q=view(h=64)), dict(h=view(b=0)), dict(ws=A + 16)):
        assert dec(**kw) == ssa.SSA_ERR_INVALID_ARG, kw
    assert dec(nb=n - 1) == ssa.SSA_ERR_WORKSPACE and dec(ws=None) == ssa.SSA_ERR_WORKSPACE

    def pre(p=p, pages=A, P=1000, nb=m):
        return ssa.ssa_prefix_decode(p, v, A, A, pages, P, A, A, v, A, A, nb, None)

    assert pre(pages=None) == ssa.SSA_ERR_INVALID_ARG
    assert pre(P=-1) == ssa.SSA_ERR_INVALID_ARG and ssa.ssa_cache_workspace_size(p, -1) == BAD
    assert pre(nb=m - 1) == ssa.SSA_ERR_WORKSPACE
    assert pre(p=cp(window=5)) == ssa.SSA_ERR_UNSUPPORTED


def test_params_from_tensors():
    q, k = torch.zeros(2, 6, 30, 64), torch.zeros(2, 3, 30, 64)
    a = ssa.window_params_for(q, k, 7, 2)
    b = ssa.window_params(2, 6, 3, 30, 64, 7, 2, torch.float32)
    assert bytes(a) == bytes(b) and isinstance(a, ssa.ssa_window_params_t)
    a = ssa.window_params_for(q.bfloat16(), k, 0, sm_scale=0.25, flags=2)
    assert (a.dtype, a.sm_scale, a.flags, a.window) == (ssa.SSA_BF16, 0.25, 2, 0)
    pool, table = torch.zeros(9, 2, 3, 16, 64, dtype=torch.bfloat16)[:, 0], torch.zeros(5, 4, dtype=torch.int32)
    a = ssa.cache_params_for(q[0], pool, table, 9, 1)
    assert bytes(a) == bytes(ssa.cache_params(5, 30, 3, 64, 16, 9, 4, torch.bfloat16, 9, 1, None, 2 * 3 * 16 * 64))
    for bad in (lambda: ssa.window_params_for(q[0], k, 7), lambda: ssa.window_params_for(q.half(), k, 7),
                lambda: ssa.cache_params_for(q, pool[0], table), lambda: ssa.cache_params_for(q, pool, table[0]),
                lambda: ssa.window_params_for(q, k, 1 << 40)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        ssa.window_params_for(q, k, "7")


def test_tensor_helpers_check_shape_type_and_device():
    t = torch.zeros(1, 2, 8, 64)
    p = ssa.window_params_for(t, t, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ssa.window_fwd(p, t, t, t)
    c = cp()
    with pytest.raises(ValueError, match="CUDA"):
        ssa.paged_decode(c, t, t, t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        ssa.cache_append(c, t, t, t, t, t, t)
    with pytest.raises(TypeError, match="tensor"):
        ssa.window_fwd(p, None, t, t)
    with pytest.raises(TypeError, match="structure"):
        ssa.window_fwd(c, t, t, t)
