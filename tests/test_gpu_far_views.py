"""Calls that the documentation allows and that reach far or twice: rows more than
2^32 elements apart, pages named more than once, one tensor for several inputs."""
import math

import pytest
import torch

import attention_ref as R
from block_sparse_full_b200 import ssa
from test_gpu_paged import _reference

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FAR = (1 << 32) + 64


@pytest.mark.parametrize("flags", [0, ssa.SSA_FLAG_FORCE_SIMT])
def test_window_rows_past_32_bits(flags):
    # the second batch entry (and, in a second layout, the second head) of every tensor lies 2^32 elements on
    T, D, H = 150, 64, 2
    g = torch.Generator().manual_seed(1)
    far = torch.empty(FAR + 5 * H * T * D + 64, dtype=torch.bfloat16, device=DEV)
    for axis in (0, 1):
        x = [torch.randn(2, H, T, D, generator=g).bfloat16() for _ in range(4)]
        n = H * T * D
        strides = (FAR, T * D, D, 1) if axis == 0 else (T * D, FAR, D, 1)
        q, k, v, dh = (far.as_strided((2, H, T, D), strides, i * n) for i in range(4))
        for a, b in zip((q, k, v, dh), x):
            a.copy_(b)
        out = {"h": far.as_strided((2, H, T, D), strides, 4 * n), "lse": torch.empty(2, H, T, device=DEV)}
        p = ssa.window_params_for(q, k, 70, 3, flags=flags)
        ssa.window_fwd(p, q, k, v, out=out)
        got = {n: t.cpu() for n, t in out.items()}
        dq = torch.empty(2, H, T, D, dtype=torch.bfloat16, device=DEV)
        dk, dv = torch.empty_like(dq), torch.empty_like(dq)
        ssa.window_bwd(p, q, k, v, out, dh, out=(dq, dk, dv))
        # gradients into the far rows too, over q, k and v once those are used up
        own = tuple(torch.empty_like(dq).copy_(t) for t in (q, k, v))
        ssa.window_bwd(p, *own, out, dh, out=(q, k, v))
        torch.cuda.synchronize()
        ssa.device_status()
        assert torch.equal(q, dq) and torch.equal(k, dk) and torch.equal(v, dv)
        ref = R.window(*x[:3], 70, 3, None, 1 / math.sqrt(D), x[3])
        R.check({**got, "dq": dq, "dk": dk, "dv": dv}, ref, ["h", "lse", "dq", "dk", "dv"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_pages_past_32_bits(dtype):
    # the prefix and the own pages at the far end of a pool of more than 2^32 elements
    Hq, Hkv, D, page, P, B = 8, 2, 128, 64, 130, 9
    n = FAR // (Hkv * page * D) + 2 + 3 + B
    kp = torch.empty(n, Hkv, page, D, dtype=DT[dtype], device=DEV)
    vp = torch.empty_like(kp)
    g = torch.Generator().manual_seed(2)
    pre = torch.tensor([n - 1, n - 3, n - 2], dtype=torch.int32)
    table = torch.arange(n - 3 - B, n - 3, dtype=torch.int32).view(B, 1)
    lens = [3, 0, 64, 1, 17, 9, 2, 30, 5]
    k, v = (torch.randn(3 + B, Hkv, page, D, generator=g).to(DT[dtype]) for _ in range(2))
    kp[-3 - B:], vp[-3 - B:] = k.to(DEV), v.to(DEV)
    q = torch.randn(B, Hq, D, generator=g).to(DT[dtype])
    p = ssa.cache_params_for(q, kp, table)
    out = ssa.prefix_decode(p, q.to(DEV), kp, vp, pre.to(DEV), P, table.to(DEV),
                            torch.tensor(lens, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    ssa.device_status()
    first = n - 3 - B

    def rows(pool, ids, m):
        return pool[[int(i) - first for i in ids]].transpose(1, 2).reshape(-1, Hkv, D)[:m]

    toks = [(rows(k, table[b], lens[b]), rows(v, table[b], lens[b]), 0) for b in range(B)]
    ref = _reference(q, toks, 0, (rows(k, pre, P), rows(v, pre, P)), 1 / math.sqrt(D), q.dtype)
    R.check(out, ref, ["h", "lse"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,P", [(3, 0), (3, 40), (12, 40)])
def test_pages_named_twice(B, P, dtype):
    # sequences that share pages, one page several times in a sequence, prefix pages among a sequence's own
    Hq, Hkv, D, page = 4, 2, 64, 16
    g = torch.Generator().manual_seed(B + P)
    kp, vp = (torch.randn(5, Hkv, page, D, generator=g).to(DT[dtype]) for _ in range(2))
    table = torch.tensor([[0, 0, 1], [1, 0, 0], [2, 3, 2]] * (B // 3), dtype=torch.int32)
    pre, lens = torch.tensor([2, 2, 4], dtype=torch.int32), [48, 33, 47] * (B // 3)
    q = torch.randn(B, Hq, D, generator=g).to(DT[dtype])
    qd, kd, vd, td, ld = (x.to(DEV) for x in (q, kp, vp, table, torch.tensor(lens, dtype=torch.int32)))
    p = ssa.cache_params_for(qd, kd, td)
    out = (ssa.prefix_decode(p, qd, kd, vd, pre.to(DEV), P, td, ld) if P else ssa.paged_decode(p, qd, kd, vd, td, ld))
    torch.cuda.synchronize()
    ssa.device_status()

    def rows(pool, ids, m):
        return pool[ids.long()].transpose(1, 2).reshape(-1, Hkv, D)[:m]

    toks = [(rows(kp, table[b], lens[b]), rows(vp, table[b], lens[b]), 0) for b in range(B)]
    ref = _reference(q, toks, 0, (rows(kp, pre, P), rows(vp, pre, P)) if P else None, 1 / math.sqrt(D), q.dtype)
    R.check(out, ref, ["h", "lse"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_tensor_for_several_inputs(dtype):
    x = torch.randn(2, 3, 200, 64, generator=torch.Generator().manual_seed(5)).to(DT[dtype])
    d = x.to(DEV)
    p = ssa.window_params_for(d, d, 50, 2)
    out = dict(ssa.window_fwd(p, d, d, d))
    out["dq"], out["dk"], out["dv"] = ssa.window_bwd(p, d, d, d, out, d)
    torch.cuda.synchronize()
    ssa.device_status()
    R.check(out, R.window(x, x, x, 50, 2, None, 1 / 8, x), ["h", "lse", "dq", "dk", "dv"])
