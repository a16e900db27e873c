"""Rows of the paged attention whose scores are not finite numbers: every plan
(one CTA, clusters, stretches joined by a second kernel, a shared prefix on
either kind of core) gives them the formula's value, and no other row changes."""
import math

import pytest
import torch

from block_sparse_full_b200 import ssa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}

# Hq, Hkv, D, page, slots of a sequence, prefix, lens, window, sinks
PLANS = {
    "one-key": (4, 2, 128, 16, 16, 0, [1, 0], 0, 0),
    "cluster": (4, 2, 64, 64, 512, 0, [300, 65, 0], 0, 0),
    "cluster-window": (4, 2, 128, 64, 4096, 0, [1500], 200, 4),
    "own-cta": (2, 1, 64, 16, 1 << 15, 0, [40] * 300, 0, 0),
    "stretches": (4, 2, 128, 64, 1 << 15, 0, [9000, 65, 0], 0, 0),
    "prefix-16-rows": (4, 2, 128, 16, 64, 500, [10, 0, 40], 0, 0),
    "prefix-128-rows": (8, 2, 64, 32, 64, 1000, [10, 0] + [33] * 10, 0, 0),
    "prefix-alone": (4, 1, 128, 64, 64, 65, [0] * 6, 0, 0),
}


def _make(plan, dtype, seed=0):
    Hq, Hkv, D, page, slots, P, lens, window, sinks = PLANS[plan]
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, need = len(lens), max(1, -(-max(lens) // page))
    shared = -(-P // page)
    n = B * need + shared
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(DT[dtype])  # noqa: E731
    kp, vp, q = rnd(n, Hkv, page, D), rnd(n, Hkv, page, D), rnd(B, Hq, D)
    table = torch.full((B, max(need, slots // page)), -1, dtype=torch.int32, device=DEV)
    table[:, :need] = torch.arange(B * need, dtype=torch.int32, device=DEV).view(B, need)
    pre = B * need + torch.arange(shared, dtype=torch.int32, device=DEV)
    lt = torch.tensor(lens, dtype=torch.int32, device=DEV)
    p = ssa.cache_params_for(q, kp, table, window, sinks, 1 / math.sqrt(D))

    def run():
        out = (ssa.prefix_decode(p, q, kp, vp, pre, P, table, lt) if P
               else ssa.paged_decode(p, q, kp, vp, table, lt))
        torch.cuda.synchronize()
        ssa.device_status()
        return out["h"].clone(), out["lse"].clone()

    return q, kp, vp, pre, run


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("plan", PLANS)
def test_query_of_nan(plan, dtype):
    # a NaN score makes the softmax NaN: h and lse of that row, and of no other
    lens, P = PLANS[plan][6], PLANS[plan][5]
    q, _, _, _, run = _make(plan, dtype)
    h0, l0 = run()
    rows = torch.zeros_like(l0, dtype=torch.bool)
    rows[0, 1] = rows[-1, 0] = rows[len(lens) // 2, -1] = True
    q[0, 1], q[-1, 0, 5], q[len(lens) // 2, -1, -1] = math.nan, math.nan, math.nan
    h, lse = run()
    empty = torch.tensor([n + P == 0 for n in lens], device=DEV)[:, None]
    bad = rows & ~empty
    assert torch.isnan(h[bad]).all() and torch.isnan(lse[bad]).all()
    assert torch.equal(h[~bad], h0[~bad]) and torch.equal(lse[~bad], l0[~bad])
    at = empty.expand_as(rows)
    assert (h[at] == 0).all() and (lse[at] == -math.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("plan", PLANS)
def test_scores_of_minus_infinity(plan, dtype):
    # every score -inf: lse = log 0 = -inf and h = 0 / 0; +inf among the scores: neither is a finite number
    lens, P = PLANS[plan][6], PLANS[plan][5]
    q, kp, _, _, run = _make(plan, dtype, 1)
    kp[..., 3] = kp[..., 3].abs() + 1
    h0, l0 = run()
    q[0, 0, 3], q[0, 1, 3] = -math.inf, math.inf
    h, lse = run()
    rows = torch.zeros_like(l0, dtype=torch.bool)
    if lens[0] + P:
        rows[0, :2] = True
        assert torch.isnan(h[0, :2]).all()
        assert lse[0, 0] == -math.inf and not torch.isfinite(lse[0, 1])
    assert torch.equal(h[~rows], h0[~rows]) and torch.equal(lse[~rows], l0[~rows])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("plan", PLANS)
def test_keys_of_nan(plan, dtype):
    # the last keys that a sequence (or the prefix) sees are NaN: all rows of that head that see them
    Hq, Hkv, D, page, slots, P, lens, window, sinks = PLANS[plan]
    q, kp, _, pre, run = _make(plan, dtype, 2)
    h0, l0 = run()
    rows, G = torch.zeros_like(l0, dtype=torch.bool), Hq // Hkv
    need = max(1, -(-max(lens) // page))
    if lens[0]:
        first = (lens[0] - 1) // page * page  # from the last page's start, its only token among them
        kp[(lens[0] - 1) // page, 0, :lens[0] - first] = math.nan
        rows[0, :G] = True
    elif P:
        kp[pre[(P - 1) // page].item(), 0] = math.nan
        rows[:, :G] = True
    h, lse = run()
    assert need and torch.isnan(h[rows]).all() and torch.isnan(lse[rows]).all()
    assert torch.equal(h[~rows], h0[~rows]) and torch.equal(lse[~rows], l0[~rows])
