"""Sliding-window attention with sinks, forward and backward, against the
float64 reference with elementwise bounds."""
import math

import pytest
import torch

import attention_ref as R
from block_sparse_full_b200 import ssa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _make(B, Hq, Hkv, T, D, dtype, rows=False, seed=0):
    g = torch.Generator().manual_seed(seed)

    def heads(H):
        x = torch.randn(B, T, H, D, generator=g).to(DT[dtype])
        return x.transpose(1, 2) if rows else x.transpose(1, 2).contiguous()

    return heads(Hq), heads(Hkv), heads(Hkv), heads(Hq)


def _dev(x):
    """On the GPU with the same strides."""
    y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=DEV)
    return y.copy_(x)


def _run(B, Hq, Hkv, T, D, dtype, window, sinks, lens=None, rows=False, grad=True, flags=0, seed=0):
    q, k, v, dh = _make(B, Hq, Hkv, T, D, dtype, rows, seed)
    lens_t = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    if lens is not None:  # what lies behind a length must not matter
        for x in (q, k, v, dh):
            for b, n in enumerate(lens):
                x[b, :, n:] = float("nan")
    scale = 1 / math.sqrt(D)
    qd, kd, vd, dhd = map(_dev, (q, k, v, dh))
    p = ssa.window_params_for(qd, kd, window, sinks, scale, flags)
    ld = None if lens is None else lens_t.to(DEV)
    out = ssa.window_fwd(p, qd, kd, vd, lens=ld)
    if grad:
        out = dict(out)
        out["dq"], out["dk"], out["dv"] = ssa.window_bwd(p, qd, kd, vd, out, dhd, lens=ld)
    torch.cuda.synchronize()
    ssa.device_status()
    ref = R.window(q, k, v, window, sinks, lens_t, scale, dh if grad else None)
    R.check(out, ref, ["h", "lse"] + (["dq", "dk", "dv"] if grad else []))
    return out


# B, Hq, Hkv, T, D, window, sinks
SHAPES = [
    (1, 1, 1, 1, 64, 0, 0),
    (1, 2, 1, 2, 128, 1, 0),
    (2, 2, 2, 63, 64, 5, 3),
    (1, 4, 2, 64, 128, 64, 0),
    (1, 3, 1, 65, 128, 64, 4),
    (1, 2, 1, 127, 128, 127, 128),
    (1, 2, 2, 128, 64, 100, 1),
    (2, 4, 1, 129, 128, 16, 4),
    (1, 1, 1, 300, 128, 0, 0),
    (1, 6, 2, 333, 64, 128, 128),
    (1, 2, 1, 511, 128, 129, 17),
    (1, 2, 1, 640, 128, 256, 64),
    (1, 2, 1, 777, 128, 200, 100),
    (2, 8, 1, 400, 64, 33, 2),
    (1, 2, 1, 1030, 128, 1, 4),
    (1, 1, 1, 1300, 128, 1000, 128),
    (1, 2, 1, 515, 64, 4096, 4),
    (2, 4, 2, 900, 128, 130, 80),  # the sinks' second tile is a 16-row step
    (1, 2, 1, 2500, 64, 40, 97),
    # few key and query tiles with long lists (clusters share them), and many
    (1, 8, 1, 700, 128, 0, 0),
    (1, 8, 1, 1500, 128, 300, 4),
    (2, 8, 2, 901, 64, 0, 0),
    (1, 16, 1, 130, 128, 0, 0),
    (1, 9, 3, 1100, 64, 700, 70),
    (3, 12, 12, 1000, 64, 260, 4),
    (1, 2, 1, 1500, 128, 0, 0),
    (1, 2, 2, 2200, 64, 1300, 100),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_window(shape, dtype):
    B, Hq, Hkv, T, D, window, sinks = shape
    _run(B, Hq, Hkv, T, D, dtype, window, sinks, seed=T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_padded_batch(dtype, D):
    # lengths of 0, 1, a tile's end and the whole; NaN behind each of them
    _run(5, 4, 2, 300, D, dtype, 70, 4, lens=[0, 1, 128, 300, 257], seed=3)
    _run(3, 2, 1, 200, D, dtype, 0, 0, lens=[199, 64, 0], rows=True, seed=4)
    _run(3, 2, 1, 1300, D, dtype, 0, 0, lens=[5, 1300, 700], seed=5)
    _run(2, 4, 1, 1700, D, dtype, 1100, 90, lens=[1601, 0], rows=True, seed=6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_token_major_layout(dtype):
    out = _run(2, 4, 2, 260, 128, dtype, 96, 4, rows=True)
    assert out["h"].stride() == (260 * 4 * 128, 128, 4 * 128, 1)
    assert out["dk"].stride() == (260 * 2 * 128, 128, 2 * 128, 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_one_projection(dtype):
    # q, k and v as slices of a fused [B, T, (Hq + 2 Hkv) D] projection
    B, Hq, Hkv, T, D = 2, 4, 2, 190, 64
    g = torch.Generator().manual_seed(9)
    x = torch.randn(B, T, (Hq + 2 * Hkv) * D, generator=g).to(DT[dtype])
    dh = torch.randn(B, Hq, T, D, generator=g).to(DT[dtype])
    xd = x.to(DEV)

    def cut(y):
        y = y.view(B, T, Hq + 2 * Hkv, D).transpose(1, 2)
        return y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]

    q, k, v = cut(xd)
    dx = torch.full_like(xd, float("nan"))
    p = ssa.window_params_for(q, k, 50, 3)
    fwd = ssa.window_fwd(p, q, k, v)
    ssa.window_bwd(p, q, k, v, fwd, dh.to(DEV), out=cut(dx))
    torch.cuda.synchronize()
    ssa.device_status()
    ref = R.window(*cut(x), 50, 3, None, 1 / math.sqrt(D), dh)
    dq, dk, dv = cut(dx)
    R.check({**fwd, "dq": dq, "dk": dk, "dv": dv}, ref, ["h", "lse", "dq", "dk", "dv"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_far_apart(dtype):
    # rows whose scores span hundreds: the running maximum moves on every tile
    T, D = 600, 128
    q, k, v, dh = _make(1, 2, 1, T, D, dtype, seed=5)
    k = (k.float() * torch.linspace(0.1, 12, T)[None, None, :, None]).to(k.dtype)
    p = ssa.window_params_for(q, k, 300, 4)
    qd, kd, vd = (x.to(DEV) for x in (q, k, v))
    out = dict(ssa.window_fwd(p, qd, kd, vd))
    out["dq"], out["dk"], out["dv"] = ssa.window_bwd(p, qd, kd, vd, out, dh.to(DEV))
    torch.cuda.synchronize()
    R.check(out, R.window(q, k, v, 300, 4, None, 1 / math.sqrt(D), dh), ["h", "lse", "dq", "dk", "dv"])


def test_equals_the_cuda_core_kernels():
    # both paths within their bounds on one padded, strided, shared-head input
    for flags in (0, ssa.SSA_FLAG_FORCE_SIMT):
        _run(2, 4, 2, 290, 128, "bf16", 77, 5, lens=[290, 133], rows=True, flags=flags, seed=11)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeatable(dtype):
    # shared heads, sinks seen by every token: the sums have a fixed order
    q, k, v, dh = (x.to(DEV) for x in _make(2, 8, 2, 1500, 128, dtype, seed=6))
    p = ssa.window_params_for(q, k, 200, 100)
    runs = []
    for _ in range(3):
        f = ssa.window_fwd(p, q, k, v)
        runs.append([f["h"], f["lse"], *ssa.window_bwd(p, q, k, v, f, dh)])
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def test_gradients_against_differences():
    # f32 gradients against central differences of the float64 reference's <dh, h>
    T, D, W, S = 40, 64, 9, 2
    q, k, v, dh = _make(1, 2, 1, T, D, "f32", seed=8)
    qd, kd, vd = (x.to(DEV) for x in (q, k, v))
    p = ssa.window_params_for(qd, kd, W, S)
    f = ssa.window_fwd(p, qd, kd, vd)
    grads = ssa.window_bwd(p, qd, kd, vd, f, dh.to(DEV))

    def loss(q, k, v):
        return (R.window(q, k, v, W, S, None, 1 / math.sqrt(D))["h"] * dh.double()).sum().item()

    base = [x.double() for x in (q, k, v)]
    g = torch.Generator().manual_seed(1)
    for i, gr in enumerate(grads):
        for _ in range(3):
            step = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
            eps = 1e-5
            hi = loss(*[x + eps * step if j == i else x for j, x in enumerate(base)])
            lo = loss(*[x - eps * step if j == i else x for j, x in enumerate(base)])
            want = (hi - lo) / (2 * eps)
            got = (gr.double().cpu() * step).sum().item()
            size = (gr.double().cpu().abs() * step.abs()).sum().item()
            assert abs(got - want) <= 1e-5 * size, (i, got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_on_another_stream(dtype):
    q, k, v, dh = (x.to(DEV) for x in _make(2, 4, 2, 500, 128, dtype, seed=12))
    lens = torch.tensor([500, 300], dtype=torch.int32, device=DEV)
    p = ssa.window_params_for(q, k, 100, 4)

    def step():
        f = ssa.window_fwd(p, q, k, v, lens=lens)
        return [f["h"], f["lse"], *ssa.window_bwd(p, q, k, v, f, dh, lens=lens)]

    want = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
        graph = torch.cuda.CUDAGraph()
    side.synchronize()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for x in held:
        x.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, other, held):
        assert torch.equal(a, b) and torch.equal(a, c)
    # new inputs and lengths in place: the captured launches follow them
    q.copy_(q.flip(2)), lens.copy_(torch.tensor([77, 0], dtype=torch.int32))
    graph.replay()
    want = step()
    torch.cuda.synchronize()
    for a, c in zip(want, held):
        assert torch.equal(a, c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_streams_at_once_with_shared_tiles(dtype):
    # few tiles with long lists: clusters of CTAs share them; two calls in flight, eager and replayed
    def make(seed):
        q, k, v, dh = map(_dev, _make(1, 4, 1, 1700, 128, dtype, False, seed))
        return ssa.window_params_for(q, k, 1300, 5), q, k, v, dh

    def both(c):
        p, q, k, v, dh = c
        out = ssa.window_fwd(p, q, k, v)
        return (out["h"], out["lse"]) + tuple(ssa.window_bwd(p, q, k, v, out, dh))

    calls = [make(1), make(2)]
    want = [both(c) for c in calls]
    streams = [torch.cuda.Stream(DEV) for _ in calls]
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


def test_length_out_of_range_is_reported():
    q, k, v, _ = (x.to(DEV) for x in _make(2, 1, 1, 100, 64, "bf16"))
    p = ssa.window_params_for(q, k, 10, 0)
    out = ssa.window_fwd(p, q, k, v, lens=torch.tensor([101, -3], dtype=torch.int32, device=DEV))
    with pytest.raises(ssa.SsaError, match="length"):
        ssa.device_status()
    ssa.device_status()  # the record was cleared
    want = ssa.window_fwd(p, q, k, v, lens=torch.tensor([100, 0], dtype=torch.int32, device=DEV))
    assert torch.equal(out["h"], want["h"])
