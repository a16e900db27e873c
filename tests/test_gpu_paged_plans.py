"""Instances of the paged cache's kernels that test_gpu_paged's shapes do not
reach: appends of many tokens and of many sequences, element-wise rotations,
the 128-row pass over a prefix with every page size."""
import pytest
import torch

from block_sparse_full_b200 import ssa
from test_gpu_paged import DEV, DT, _freq, test_append as _append_case, test_prefix_decode as _prefix_case

pytestmark = pytest.mark.gpu


def _counts(n, per, empty):
    return [0 if b in empty else 1 + (b * 7 + n) % per for b in range(n)]


def _lens(n, page):
    return [(b * 5) % (2 * page + 1) for b in range(n)]


APPEND = [
    # B, Hq, Hkv, D, page, counts, lens, rot, interleaved: more than 512 rows
    (1, 2, 1, 64, 32, [700], [13], 64, False),
    (3, 4, 2, 128, 16, [200, 1, 400], [0, 15, 16], 128, True),
    (2, 3, 1, 64, 64, [290, 300], [1, 64], 24, False),
    (2, 2, 2, 64, 16, [513, 0], [5, 3], 20, False),      # half of 10: one element at a time
    (2, 2, 1, 128, 32, [1, 530], [31, 0], 22, True),     # pair by pair
    (2, 1, 1, 64, 16, [300, 301], [0, 1], 0, False),
    # the search past 31 sequences, empty ones at its turns
    (31, 1, 1, 64, 16, _counts(31, 5, {0, 30}), _lens(31, 16), 64, False),
    (32, 2, 1, 64, 16, _counts(32, 9, {30, 31}), _lens(32, 16), 22, True),
    (33, 2, 1, 64, 32, _counts(33, 30, {31, 32}), _lens(33, 32), 64, True),
    (64, 1, 1, 128, 16, _counts(64, 20, {0, 31, 32, 33, 62, 63}), _lens(64, 16), 128, False),
    (70, 2, 1, 64, 16, _counts(70, 20, set(range(29, 36)) | {64, 69}), _lens(70, 16), 20, False),
    (70, 4, 2, 64, 64, _counts(70, 4, {1, 63, 64, 65}), _lens(70, 64), 6, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"B{c[0]}-N{sum(c[5])}-rot{c[7]}-{c[8]}")
def test_append(case, dtype):
    _append_case(case, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot,inter", [(20, False), (22, True), (18, False), (2, True)])
def test_append_rotations_of_odd_halves(rot, inter, dtype):
    _append_case((3, 3, 1, 64, 16, [5, 0, 14], [40, 9, 3], rot, inter), dtype)


@pytest.mark.parametrize("n", [1, 3, 60])
def test_equal_shares_are_the_ranges_that_say_so(n):
    # without q_start: one, a few and (together above 512) many tokens each, lengths apart and in place
    B, Hq, Hkv, D, page = 35, 2, 1, 64, 16
    g = torch.Generator(device=DEV).manual_seed(n)
    q, k, v = (torch.randn(B * n, H, D, generator=g, device=DEV).bfloat16() for H in (Hq, Hkv, Hkv))
    width = 8
    table = torch.randperm(B * width, generator=g, device=DEV).to(torch.int32).view(B, width)
    lens = (torch.arange(B, device=DEV) * 3 % 60).to(torch.int32)
    start = (torch.arange(B + 1, device=DEV) * n).to(torch.int32)
    f = _freq(D).to(DEV)
    got = []
    for how in range(3):
        kp, vp = (torch.zeros(B * width, Hkv, page, D, dtype=DT["bf16"], device=DEV) for _ in range(2))
        p, l = ssa.cache_params_for(q, kp, table), lens.clone()
        out = ssa.cache_append(p, kp, vp, table, l, k, v, q=q, inv_freq=f, q_start=start if how == 0 else None,
                               new_lens=l if how == 2 else None)
        got.append((out["q"], out["lens"], kp, vp))
    torch.cuda.synchronize()
    ssa.device_status()
    assert torch.equal(got[0][1], lens + n)
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


PREFIX = [
    # Hq, Hkv, D, page, prefix, lens: more than 16 rows a head
    (8, 2, 128, 32, 1000, [10] * 17),
    (6, 2, 128, 128, 700, [3, 0, 130] * 4),
    (4, 1, 64, 128, 1111, [1, 200, 0, 64, 65] * 2),
    (2, 1, 64, 32, 777, [7] * 33),
    (8, 1, 128, 128, 65, [2, 0, 1]),
    (8, 1, 128, 128, 129, [2, 0, 1]),
    (3, 1, 64, 16, 47, [5] * 50),             # row tiles of 126 rows
    (4, 1, 128, 32, 4100, [9] * 70),          # two row tiles and two more rows
    (130, 1, 64, 16, 200, [5, 0]),            # a group of more rows than a row tile
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", PREFIX, ids=str)
def test_prefix_decode(case, dtype):
    _prefix_case(case, dtype)
