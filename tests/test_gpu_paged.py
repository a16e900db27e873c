"""The paged cache: appending with rotation, and the attention of single tokens
over it, alone and behind a shared prefix, against float64 references."""
import math

import pytest
import torch

import attention_ref as R
from block_sparse_full_b200 import ssa

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _freq(rot):
    return None if rot == 0 else 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _pool(B, Hkv, D, page, width, dtype, seed, shared=0, spare=2):
    """Pages full of NaN, a shuffled table, the shared pages."""
    g = torch.Generator().manual_seed(seed)
    n = B * width + shared + spare
    order = torch.randperm(n, generator=g).to(torch.int32)
    pages = torch.full((n, Hkv, page, D), float("nan"), dtype=DT[dtype])
    return pages, pages.clone(), order[:B * width].view(B, width).contiguous(), order[B * width:B * width + shared].contiguous()


# ------------------------------------------------------------------ append

APPEND = [
    # B, Hq, Hkv, D, page, counts, lens, rot, interleaved
    (1, 1, 1, 64, 16, [1], [0], 64, False),
    (3, 4, 2, 128, 16, [1, 1, 1], [0, 15, 16], 128, False),
    (2, 2, 2, 64, 32, [5, 40], [31, 7], 32, True),
    (4, 6, 1, 128, 64, [0, 130, 1, 63], [5, 0, 63, 64], 24, False),
    (2, 3, 3, 64, 128, [7, 9], [127, 128], 20, True),
    (2, 8, 4, 128, 16, [33, 2], [100000, 131000], 128, True),
    (2, 2, 1, 64, 64, [4, 4], [0, 9], 0, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append(case, dtype):
    B, Hq, Hkv, D, page, counts, lens, rot, inter = case
    behind = 3
    N = sum(counts) + behind
    g = torch.Generator().manual_seed(N + rot)
    q, k, v = (torch.randn(N, H, D, generator=g).to(DT[dtype]) for H in (Hq, Hkv, Hkv))
    width = max((n + c + page - 1) // page for n, c in zip(lens, counts))
    small = width > 100  # far positions: all but the last pages of a sequence are one page
    kp, vp, table, _ = _pool(B, Hkv, D, page, 8 if small else width, dtype, 1)
    if small:
        near = table
        table = torch.zeros(B, width, dtype=torch.int32)
        for b in range(B):
            first = lens[b] // page
            table[b, first:first + 8] = near[b, :len(table[b, first:first + 8])]
    start = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0).to(torch.int32)
    lens_t = torch.tensor(lens, dtype=torch.int32)
    f = _freq(rot)
    qd, kd, vd, kpd, vpd = (x.to(DEV) for x in (q, k, v, kp, vp))
    p = ssa.cache_params_for(qd, kpd, table)
    k_out = torch.empty_like(kd)
    out = ssa.cache_append(p, kpd, vpd, table.to(DEV), lens_t.to(DEV), kd, vd, q=qd,
                           inv_freq=None if f is None else f.to(DEV), interleaved=inter, q_start=start.to(DEV),
                           k_out=k_out)
    torch.cuda.synchronize()
    ssa.device_status()
    assert out["lens"].tolist() == [n + c for n, c in zip(lens, counts)]
    used = sum(counts)
    pos = torch.cat([torch.arange(n, n + c) for n, c in zip(lens, counts)]) if used else torch.zeros(0)
    for x, got in ((q, out["q"].cpu()), (k, k_out.cpu())):
        want = R.rotate(x[:used].double(), pos, f, inter)
        assert ((got[:used].double() - want).abs() <= R.rotate_tol(x[:used], x.dtype)).all()
        if rot < D:
            assert torch.equal(got[:used, :, rot:], x[:used, :, rot:])
        assert torch.equal(got[used:], x[used:])  # rows behind the last sequence
    kp2, vp2 = kpd.cpu(), vpd.cpu()
    i = 0
    for b in range(B):
        for j in range(counts[b]):
            slot = lens[b] + j
            pg, off = int(table[b, slot // page]), slot % page
            assert torch.equal(kp2[pg, :, off], k_out[i].cpu()) and torch.equal(vp2[pg, :, off], v[i])
            kp2[pg, :, off], vp2[pg, :, off] = float("nan"), float("nan")
            i += 1
    assert torch.isnan(kp2).all() and torch.isnan(vp2).all()  # nothing else was written


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_in_place_and_strided(dtype):
    # q, k, v as slices of one projection, rotated where they lie; lengths advanced in place;
    # pages of keys and values side by side in one pool
    B, Hq, Hkv, D, page, n = 3, 4, 2, 64, 16, 5
    g = torch.Generator().manual_seed(2)
    x = torch.randn(B * n, (Hq + 2 * Hkv) * D, generator=g).to(DT[dtype])
    xd = x.to(DEV)
    rows = xd.view(B * n, -1, D)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    pool = torch.zeros(B * 2, 2, Hkv, page, D, dtype=DT[dtype], device=DEV)
    table = torch.arange(B * 2, dtype=torch.int32, device=DEV).view(B, 2)
    lens = torch.tensor([0, 13, 27], dtype=torch.int32, device=DEV)
    f = _freq(D)
    p = ssa.cache_params_for(q, pool[:, 0], table)
    out = ssa.cache_append(p, pool[:, 0], pool[:, 1], table, lens, k, v, q=q, inv_freq=f.to(DEV), new_lens=lens,
                           q_out=q, k_out=k, pos_offset=7)
    torch.cuda.synchronize()
    ssa.device_status()
    assert out["q"] is q and lens.tolist() == [5, 18, 32]
    pos = torch.cat([torch.arange(s, s + n) for s in (7, 20, 34)])
    was = x.view(B * n, -1, D)
    want = R.rotate(was[:, :Hq + Hkv].double(), pos, f, False)
    now = rows.cpu()
    assert ((now[:, :Hq + Hkv].double() - want).abs() <= R.rotate_tol(was[:, :Hq + Hkv], x.dtype)).all()
    assert torch.equal(now[:, Hq + Hkv:], was[:, Hq + Hkv:])
    flat = pool.cpu().permute(1, 0, 3, 2, 4).reshape(2, B, 2 * page, Hkv, D)
    for b, s in enumerate((0, 13, 27)):
        assert torch.equal(flat[0, b, s:s + n], now[b * n:(b + 1) * n, Hq:Hq + Hkv])
        assert torch.equal(flat[1, b, s:s + n], now[b * n:(b + 1) * n, Hq + Hkv:])


def test_append_past_the_end_is_reported():
    B, Hkv, D, page = 2, 1, 64, 16
    pool = torch.zeros(4, Hkv, page, D, device=DEV)
    vpool = pool.clone()
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32, device=DEV)  # page 9 does not exist
    k = torch.ones(6, Hkv, D, device=DEV)
    p = ssa.cache_params_for(k, pool, table)
    lens = torch.tensor([30, 15], dtype=torch.int32, device=DEV)
    out = ssa.cache_append(p, pool, vpool, table, lens, k, k)
    with pytest.raises(ssa.SsaError, match="out of range"):
        ssa.device_status()
    ssa.device_status()
    assert out["lens"].tolist() == [32, 18]
    assert pool.sum().item() == 3 * D and pool[1, 0, 14:].sum() == 2 * D and pool[2, 0, 15].sum() == D
    # no tokens at all: lengths only
    e = torch.empty(0, Hkv, D, device=DEV)
    assert ssa.cache_append(p, pool, vpool, table, lens, e, e)["lens"].tolist() == [30, 15]


def test_offsets_past_32_bits():
    # a pool of more than 2^32 elements: its last page is written and read where it lies
    Hkv, D, page = 8, 128, 128
    n = (1 << 32) // (Hkv * D * page) + 2
    kp = torch.empty(n, Hkv, page, D, dtype=torch.bfloat16, device=DEV)
    vp = torch.empty_like(kp)
    for pool in (kp, vp):
        pool[:3].zero_(), pool[-2:].zero_()
    table = torch.tensor([[n - 1, n - 2], [1, 2]], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(260, H, D, generator=g).bfloat16().to(DEV) for H in (8, 8, 8))
    p = ssa.cache_params_for(q, kp, table)
    lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    lens = ssa.cache_append(p, kp, vp, table, lens, k, v)["lens"]
    out = ssa.paged_decode(p, q[[129, 259]], kp, vp, table, lens)
    torch.cuda.synchronize()
    ssa.device_status()
    assert torch.equal(kp[n - 1], k[:128].transpose(0, 1)) and torch.equal(vp[n - 2, :, :2], v[128:130].transpose(0, 1))
    for b in range(2):
        for h in range(8):
            a = R.attend(q[129 + 130 * b, h:h + 1].double().cpu(), k[130 * b:130 * b + 130, h].double().cpu(),
                         v[130 * b:130 * b + 130, h].double().cpu(), torch.ones(1, 130, dtype=torch.bool),
                         1 / math.sqrt(D), torch.bfloat16)
            R.check({"h": out["h"][b, h][None], "lse": out["lse"][b, h][None]}, a, ["h", "lse"])


# ------------------------------------------------------------------ attention over the pages

def _fill(kp, vp, table, lens, Hkv, D, page, dtype, g, window=0, sinks=0):
    """Random tokens in the slots that are seen (the rest stays NaN); pages that hold none of them get
    a table entry that does not exist."""
    toks = []
    for b, n in enumerate(lens):
        k, v = (torch.randn(n, Hkv, D, generator=g).to(DT[dtype]) for _ in range(2))
        w0 = max(0, n - window) if window else 0
        live = [s for s in range(n) if s >= w0 or s < sinks]
        for s in live:
            pg = int(table[b, s // page])
            kp[pg, :, s % page], vp[pg, :, s % page] = k[s], v[s]
        used = {s // page for s in live}
        for i in range(table.shape[1]):
            if i not in used:
                table[b, i] = -5
        toks.append((k, v, w0))
    return toks


def _reference(q, toks, sinks, prefix, scale, dtype):
    B, Hq, D = q.shape
    out = {"h": torch.zeros(B, Hq, D, dtype=torch.float64), "lse": torch.zeros(B, Hq, dtype=torch.float64)}
    out["h_tol"], out["lse_tol"] = torch.zeros_like(out["h"]), torch.zeros_like(out["lse"])
    for b in range(B):
        k, v, w0 = toks[b]
        s = torch.arange(k.shape[0])
        keep = (s >= w0) | (s < sinks)
        if prefix is not None:
            k, v = torch.cat([prefix[0], k]), torch.cat([prefix[1], v])
            keep = torch.cat([torch.ones(prefix[0].shape[0], dtype=torch.bool), keep])
        G = Hq // k.shape[1]
        for h in range(Hq):
            a = R.attend(q[b, h:h + 1].double(), k[:, h // G].double(), v[:, h // G].double(), keep[None], scale, dtype)
            for n in out:
                out[n][b, h] = a[n][0]
    return out


DECODE = [
    # Hq, Hkv, D, page, lens, window, sinks
    (1, 1, 64, 16, [1], 0, 0),
    (4, 1, 128, 16, [0, 1, 2, 17], 0, 0),
    (4, 2, 64, 32, [31, 32, 33, 64, 65], 0, 0),
    (8, 8, 128, 64, [300, 5], 0, 0),
    (16, 1, 128, 128, [257], 0, 0),
    (24, 1, 64, 16, [100, 63], 0, 0),          # more rows than one row tile
    (40, 1, 128, 64, [129], 0, 0),
    (4, 2, 128, 64, [1000, 40], 1, 0),
    (4, 2, 128, 16, [1000, 41, 17], 16, 4),
    (6, 2, 64, 16, [500, 130, 0], 100, 128),   # sinks and window touch or overlap
    (2, 1, 128, 32, [700, 228, 229, 100], 100, 128),
    (8, 2, 128, 64, [3000, 64, 1500, 2999, 1], 0, 0),
    (8, 2, 64, 128, [4000], 1024, 4),
    (5, 5, 128, 16, [77] * 40, 0, 0),          # more sequences than a warp
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", DECODE, ids=str)
def test_paged_decode(case, dtype):
    _decode_case(case, dtype, 0)


# The same over tables wide enough that the work is cut by the lengths, not by rows; more rows, and
# more windows, than the clusters of one launch take.
WIDE = [
    (4, 2, 128, 16, [500, 41, 17] * 50, 16, 4),
    (2, 1, 64, 64, [9000], 8500, 4),
    (8, 8, 64, 32, [5000, 0, 3], 0, 0),
    (2, 2, 128, 128, [1] * 200, 0, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", DECODE + WIDE, ids=str)
def test_paged_decode_wide_table(case, dtype):
    _decode_case(case, dtype, 1 << 15)


def _decode_case(case, dtype, slots):
    Hq, Hkv, D, page, lens, window, sinks = case
    B, g = len(lens), torch.Generator().manual_seed(sum(lens))
    width = max(1, -(-max(lens) // page))
    kp, vp, table, _ = _pool(B, Hkv, D, page, width, dtype, 5)
    toks = _fill(kp, vp, table, lens, Hkv, D, page, dtype, g, window, sinks)
    q = torch.randn(B, Hq, D, generator=g).to(DT[dtype])
    scale = 1 / math.sqrt(D)
    if slots:  # (entries behind the lengths are not read)
        table = torch.cat([table, torch.full((B, max(0, slots // page - width)), -1, dtype=torch.int32)], 1)
    qd, kpd, vpd, td = (x.to(DEV) for x in (q, kp, vp, table))
    p = ssa.cache_params_for(qd, kpd, td, window, sinks, scale)
    out = ssa.paged_decode(p, qd, kpd, vpd, td, torch.tensor(lens, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    ssa.device_status()
    R.check(out, _reference(q, toks, sinks if window else 0, None, scale, q.dtype), ["h", "lse"])


PREFIX = [
    # Hq, Hkv, D, page, prefix, lens
    (1, 1, 64, 16, 1, [0]),
    (4, 2, 128, 16, 0, [5, 0]),
    (4, 1, 128, 64, 64, [0, 0, 0]),
    (4, 2, 64, 32, 100, [1, 33, 0, 70, 64]),
    (8, 2, 128, 16, 1000, [10] * 17),
    (6, 2, 128, 128, 700, [300, 1, 129]),
    (2, 2, 64, 64, 129, [7] * 70),
    (40, 1, 128, 64, 333, [20, 0, 65, 1]),
    (3, 1, 64, 16, 4000, [50, 3]),
    (16, 2, 128, 64, 2050, list(range(64))),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", PREFIX, ids=str)
def test_prefix_decode(case, dtype):
    Hq, Hkv, D, page, P, lens = case
    B, g = len(lens), torch.Generator().manual_seed(P)
    width, shared = max(1, -(-max(lens) // page)), -(-P // page)
    kp, vp, table, pre = _pool(B, Hkv, D, page, width, dtype, 6, shared)
    toks = _fill(kp, vp, table, lens, Hkv, D, page, dtype, g)
    pk, pv = (torch.randn(P, Hkv, D, generator=g).to(DT[dtype]) for _ in range(2))
    for s in range(P):
        pg = int(pre[s // page])
        kp[pg, :, s % page], vp[pg, :, s % page] = pk[s], pv[s]
    q = torch.randn(B, Hq, D, generator=g).to(DT[dtype])
    scale = 1 / math.sqrt(D)
    qd, kpd, vpd, td = (x.to(DEV) for x in (q, kp, vp, table))
    p = ssa.cache_params_for(qd, kpd, td, 0, 0, scale)
    out = ssa.prefix_decode(p, qd, kpd, vpd, pre.to(DEV), P, td, torch.tensor(lens, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    ssa.device_status()
    R.check(out, _reference(q, toks, 0, (pk, pv), scale, q.dtype), ["h", "lse"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_scores(dtype):
    # scores that reach into the hundreds, growing along the sequence
    B, Hq, Hkv, D, page, n = 1, 4, 2, 128, 16, 700
    g = torch.Generator().manual_seed(7)
    kp, vp, table, _ = _pool(B, Hkv, D, page, 44, dtype, 8)
    k = (torch.randn(n, Hkv, D, generator=g) * torch.linspace(0.1, 15, n)[:, None, None]).to(DT[dtype])
    v = torch.randn(n, Hkv, D, generator=g).to(DT[dtype])
    for s in range(n):
        kp[table[0, s // page], :, s % page], vp[table[0, s // page], :, s % page] = k[s], v[s]
    q = torch.randn(B, Hq, D, generator=g).to(DT[dtype])
    qd, kpd, vpd, td = (x.to(DEV) for x in (q, kp, vp, table))
    p = ssa.cache_params_for(qd, kpd, td)
    out = ssa.paged_decode(p, qd, kpd, vpd, td, torch.tensor([n], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    R.check(out, _reference(q, [(k, v, 0)], 0, None, 1 / math.sqrt(D), q.dtype), ["h", "lse"])


def test_slices_of_index_arrays():
    # table, lengths, prefix pages, token ranges and lse inside larger arrays, 4 bytes off any wider alignment
    B, Hq, Hkv, D, page, P = 3, 4, 2, 64, 16, 37
    g = torch.Generator().manual_seed(4)
    ints = torch.arange(64, dtype=torch.int32, device=DEV)
    kp = torch.randn(16, Hkv, page, D, generator=g).bfloat16().to(DEV)
    vp = torch.randn(16, Hkv, page, D, generator=g).bfloat16().to(DEV)
    table, pre = ints[1:7].view(3, 2), ints[9:12]
    some = torch.tensor([99, 20, 1, 32, 99, 0, 1, 2, 3], dtype=torch.int32, device=DEV)
    lens, start = some[1:4], some[5:9]
    q = torch.randn(B, Hq, D, generator=g).bfloat16().to(DEV)
    p = ssa.cache_params_for(q, kp, table)
    lse = torch.empty(B * Hq + 1, device=DEV)
    out = {"h": torch.empty_like(q), "lse": lse[1:].view(B, Hq)}
    want = ssa.prefix_decode(p, q, kp, vp, pre.clone(), P, table.clone(), lens.clone())
    ssa.prefix_decode(p, q, kp, vp, pre, P, table, lens, out=out)
    k = torch.randn(B, Hkv, D, generator=g).bfloat16().to(DEV)
    new = ssa.cache_append(p, kp, vp, table, lens - 1, k, k, q_start=start, inv_freq=_freq(66).to(DEV)[1:])["lens"]
    torch.cuda.synchronize()
    ssa.device_status()
    assert torch.equal(out["h"], want["h"]) and torch.equal(out["lse"], want["lse"])
    assert new.tolist() == [20, 1, 32]


def test_bad_lengths_and_pages_are_reported():
    B, Hq, Hkv, D, page = 2, 2, 1, 64, 16
    pool = torch.zeros(3, Hkv, page, D, dtype=torch.bfloat16, device=DEV)
    q = torch.ones(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    table = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    p = ssa.cache_params_for(q, pool, table)
    for lens, t in (([17, 4], table), ([-1, 4], table), ([16, 16], torch.full_like(table, 3))):
        ssa.paged_decode(p, q, pool, pool, t, torch.tensor(lens, dtype=torch.int32, device=DEV))
        with pytest.raises(ssa.SsaError, match="out of range"):
            ssa.device_status()
        ssa.device_status()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix", [0, 40])
def test_prompt_then_captured_steps(dtype, prefix):
    """A prompt appended, attended with window attention, then single tokens through one captured
    step that appends and attends; every output equals attention over the tokens so far."""
    B, Hq, Hkv, D, page = 2, 4, 2, 128, 16
    W, S = (0, 0) if prefix else (24, 3)
    steps, n0 = 6, 45
    g = torch.Generator().manual_seed(13)
    f = _freq(D).to(DEV)
    c = ssa.PagedCache(B, Hq, Hkv, D, 96, DT[dtype], DEV, page=page, window=W, sinks=S, inv_freq=f, prefix_len=prefix)
    new = lambda n, H: torch.randn(n, H, D, generator=g).to(DT[dtype]).to(DEV)  # noqa: E731
    past_k, past_v = [[] for _ in range(B)], [[] for _ in range(B)]
    if prefix:
        pk, pv, turned = new(prefix, Hkv), new(prefix, Hkv), torch.empty(prefix, Hkv, D, dtype=DT[dtype], device=DEV)
        c.fill_prefix(pk, pv, k_out=turned)
        for b in range(B):
            past_k[b].append(turned), past_v[b].append(pv)
    q, k, v = new(B * n0, Hq), new(B * n0, Hkv), new(B * n0, Hkv)
    k_out = torch.empty_like(k)
    q_rot = c.append(k, v, q, k_out=k_out)
    for b in range(B):
        past_k[b].append(k_out[b * n0:(b + 1) * n0].clone()), past_v[b].append(v[b * n0:(b + 1) * n0])
    if not prefix:  # the prompt itself
        shape = lambda x, H: x.view(B, n0, H, D).transpose(1, 2)  # noqa: E731
        p = ssa.window_params(B, Hq, Hkv, n0, D, W, S, DT[dtype])
        out = ssa.window_fwd(p, shape(q_rot, Hq), shape(k_out, Hkv), shape(v, Hkv))
        torch.cuda.synchronize()
        ref = R.window(shape(q_rot, Hq).cpu(), shape(k_out, Hkv).cpu(), shape(v, Hkv).cpu(), W, S, None, 1 / math.sqrt(D))
        R.check(out, ref, ["h", "lse"])
    qs, ks, vs = new(B, Hq), new(B, Hkv), new(B, Hkv)
    qo, ko = torch.empty_like(qs), torch.empty_like(ks)

    def step():
        c.append(ks, vs, qs, q_out=qo, k_out=ko)
        return c.attend(qo)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    held = c.lens.clone()
    with torch.cuda.stream(side):
        step()  # first use outside the capture
    side.synchronize()
    c.lens.copy_(held)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for i in range(steps):
        qs.copy_(new(B, Hq)), ks.copy_(new(B, Hkv)), vs.copy_(new(B, Hkv))
        graph.replay()
        torch.cuda.synchronize()
        ssa.device_status()
        assert c.lens.tolist() == [n0 + i + 1] * B
        for b in range(B):
            past_k[b].append(ko[b:b + 1].clone()), past_v[b].append(vs[b:b + 1].clone())
        toks = []
        for b in range(B):
            kk, vv = torch.cat(past_k[b]).cpu(), torch.cat(past_v[b]).cpu()
            toks.append((kk, vv, max(0, kk.shape[0] - W) if W else 0))
        R.check(out, _reference(qo.cpu(), toks, S, None, 1 / math.sqrt(D), DT[dtype]), ["h", "lse"])


def test_decode_is_repeatable_and_shares_no_state():
    # the same call twice, and two calls on two streams at once with a workspace each
    B, Hq, Hkv, D, page = 7, 8, 2, 128, 64
    g = torch.Generator(device=DEV).manual_seed(3)
    pool = torch.randn(B * 20, Hkv, page, D, generator=g, device=DEV).bfloat16()
    vpool = torch.randn(B * 20, Hkv, page, D, generator=g, device=DEV).bfloat16()
    table = torch.randperm(B * 20, generator=g, device=DEV).to(torch.int32).view(B, 20)
    lens = torch.tensor([1280, 3, 700, 1, 0, 1279, 64], dtype=torch.int32, device=DEV)
    q = torch.randn(B, Hq, D, generator=g, device=DEV).bfloat16()
    p = ssa.cache_params_for(q, pool, table)
    a = ssa.paged_decode(p, q, pool, vpool, table, lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(ssa.paged_decode(p, q, pool, vpool, table, lens))
    torch.cuda.synchronize()
    for b in got:
        assert torch.equal(a["h"], b["h"]) and torch.equal(a["lse"], b["lse"])


def test_tensors_are_checked():
    B, Hq, Hkv, D, page = 2, 4, 2, 64, 16
    pool = torch.zeros(4, Hkv, page, D, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(B, 2, dtype=torch.int32, device=DEV)
    lens = torch.ones(B, dtype=torch.int32, device=DEV)
    q = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    k = q[:, :Hkv]
    p = ssa.cache_params_for(q, pool, table)

    def bad(what, fn, *args, **kw):
        with pytest.raises(ValueError, match=what):
            fn(p, *args, **kw)

    dec = ssa.paged_decode
    bad("q must have shape", dec, q[:1], pool, pool, table, lens)
    bad("q must be", dec, q.float(), pool, pool, table, lens)
    bad("last axis", dec, q.transpose(1, 2).contiguous().transpose(1, 2), pool, pool, table, lens)
    bad("k_pages", dec, q, pool.float(), pool, table, lens)
    bad("v_pages: each page", dec, q, pool, pool.transpose(1, 2).contiguous().transpose(1, 2), table, lens)
    bad("table must have", dec, q, pool, pool, table[:, :1], lens)
    bad("table must be", dec, q, pool, pool, table.long(), lens)
    bad("table must be contiguous", dec, q, pool, pool, table.t().contiguous().t(), lens)
    bad("lens must be", dec, q, pool, pool, table, lens.cpu())
    bad("ws must be", dec, q, pool, pool, table, lens, ws=torch.empty(1 << 20, dtype=torch.uint8))
    bad("prefix_pages", ssa.prefix_decode, q, pool, pool, table, 17, table, lens)
    bad("prefix_len", ssa.prefix_decode, q, pool, pool, table, -1, table, lens)
    app = ssa.cache_append
    bad("v must have", app, pool, pool, table, lens, k, q)
    bad("q_out without", app, pool, pool, table, lens, k, k, q_out=q)
    bad("inv_freq has more", app, pool, pool, table, lens, k, k, inv_freq=torch.ones(33, dtype=torch.float64, device=DEV))
    bad("inv_freq must be", app, pool, pool, table, lens, k, k, inv_freq=torch.ones(8, device=DEV))
    bad("q_start must have", app, pool, pool, table, lens, k, k, q_start=lens)
    bad("pos_offset", app, pool, pool, table, lens, k, k, pos_offset=-1)
    with pytest.raises(ssa.SsaError, match="new_lens overlaps"):
        big = torch.zeros(3, dtype=torch.int32, device=DEV)
        app(p, pool, pool, table, big[:2], k, k, new_lens=big[1:])
    with pytest.raises(ssa.SsaError, match="workspace"):
        dec(p, q, pool, pool, table, lens, ws=torch.empty(256, dtype=torch.uint8, device=DEV))
    w = ssa.window_params(1, 2, 1, 8, 64, 4, 0, torch.bfloat16)
    x, y = (torch.zeros(1, H, 8, 64, dtype=torch.bfloat16, device=DEV) for H in (2, 1))
    with pytest.raises(ValueError, match="k must have"):
        ssa.window_fwd(w, x, x, y)
    with pytest.raises(ssa.SsaError, match="batch stride|token stride"):
        ssa.window_fwd(w, x, y[:, :, :1].expand(1, 1, 8, 64), y)
    f = ssa.window_fwd(w, x, y, y)
    with pytest.raises(ValueError, match="dh must have"):
        ssa.window_bwd(w, x, y, y, f, y)
    with pytest.raises(ValueError, match="lse must be"):
        ssa.window_bwd(w, x, y, y, {**f, "lse": f["lse"].double()}, x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_queries_and_outputs(dtype):
    # queries as slices of a fused projection, outputs into another strided buffer
    B, Hq, Hkv, D, page, n = 3, 6, 2, 64, 32, 90
    g = torch.Generator().manual_seed(21)
    kp, vp, table, _ = _pool(B, Hkv, D, page, 3, dtype, 22)
    lens = [90, 1, 33]
    toks = _fill(kp, vp, table, lens, Hkv, D, page, dtype, g)
    x = torch.randn(B, (Hq + 2 * Hkv) * D, generator=g).to(DT[dtype])
    q = x.view(B, -1, D)[:, :Hq]
    xd, kpd, vpd, td = (t.to(DEV) for t in (x, kp, vp, table))
    qd = xd.view(B, -1, D)[:, :Hq]
    buf = torch.full((B, 2 * Hq, D), 7.0, dtype=DT[dtype], device=DEV)
    out = {"h": buf[:, ::2], "lse": torch.empty(B, Hq, device=DEV)}
    p = ssa.cache_params_for(qd, kpd, td)
    ssa.paged_decode(p, qd, kpd, vpd, td, torch.tensor(lens, dtype=torch.int32, device=DEV), out=out)
    torch.cuda.synchronize()
    ssa.device_status()
    R.check(out, _reference(q, toks, 0, None, 1 / math.sqrt(D), q.dtype), ["h", "lse"])
    assert (buf[:, 1::2] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefix_pass_captured(dtype):
    # a batch large enough for the 128-row pass, captured; replays follow the lengths, and two
    # graphs of one cache on two streams do not disturb each other
    B, Hq, Hkv, D, page, P = 20, 8, 2, 128, 16, 300
    c = ssa.PagedCache(B, Hq, Hkv, D, 64, DT[dtype], DEV, page=page, prefix_len=P)
    g = torch.Generator(device=DEV).manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(DT[dtype])  # noqa: E731
    c.fill_prefix(rnd(P, Hkv, D), rnd(P, Hkv, D))
    c.append(rnd(B * 40, Hkv, D), rnd(B * 40, Hkv, D))
    q = rnd(B, Hq, D)
    want = c.attend(q)
    side = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for s in side:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            outs.append(c.attend(q))
        graphs.append(gr)
    torch.cuda.synchronize()
    for _ in range(4):
        for s, gr in zip(side, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o["h"], want["h"]) and torch.equal(o["lse"], want["lse"])
    c.lens.copy_(torch.arange(B, dtype=torch.int32, device=DEV))
    graphs[0].replay()
    want = c.attend(q)
    torch.cuda.synchronize()
    ssa.device_status()
    assert torch.equal(outs[0]["h"], want["h"])


def test_first_calls_inside_a_capture():
    # every call captured before it has ever run in the process: nothing in it synchronises
    import subprocess
    import sys

    code = """
import torch
from block_sparse_full_b200 import ssa
for dt in (torch.bfloat16, torch.float32):
    q = torch.randn(2, 20, 4, 64, device="cuda", dtype=dt).transpose(1, 2)
    k = torch.randn(2, 20, 2, 64, device="cuda", dtype=dt).transpose(1, 2)
    p = ssa.window_params_for(q, k, 7, 2)
    c = ssa.PagedCache(20, 4, 2, 64, 40, dt, "cuda", page=16, prefix_len=20)
    x, y = torch.randn(20, 4, 64, device="cuda", dtype=dt), torch.randn(20, 2, 64, device="cuda", dtype=dt)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f = ssa.window_fwd(p, q, k, k)
        grads = ssa.window_bwd(p, q, k, k, f, q)
        c.append(y, y, x)
        out = c.attend(x)
    g.replay()
    torch.cuda.synchronize()
    ssa.device_status()
    want = ssa.window_fwd(p, q, k, k)
    assert torch.equal(f["h"], want["h"]) and c.lens.tolist() == [1] * 20
    for a, b in zip(grads, ssa.window_bwd(p, q, k, k, want, q)):
        assert torch.equal(a, b)
    assert torch.equal(out["h"], c.attend(x)["h"])
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_short_wait_limit_leaves_the_context_usable():
    # the tensor-core kernels' waits give up after 100 ns: the calls end, are reported, and later
    # calls give the same results as before
    g = torch.Generator(device=DEV).manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
    q, k, v, dh = rnd(2, 4, 700, 128), rnd(2, 2, 700, 128), rnd(2, 2, 700, 128), rnd(2, 4, 700, 128)
    c = ssa.PagedCache(20, 4, 2, 128, 64, torch.bfloat16, DEV, prefix_len=500)
    c.fill_prefix(rnd(500, 2, 128), rnd(500, 2, 128))
    c.append(rnd(100, 2, 128), rnd(100, 2, 128))
    x = rnd(20, 4, 128)

    def all_calls(window):
        p = ssa.window_params_for(q, k, window, 5)
        f = ssa.window_fwd(p, q, k, v)
        return [f["h"], f["lse"], *ssa.window_bwd(p, q, k, v, f, dh), *c.attend(x).values()]

    want = {w: all_calls(w) for w in (100, 300)}
    torch.cuda.synchronize()
    ssa.device_status()
    stream = torch.cuda.current_stream().cuda_stream
    for w in (100, 300):
        ssa.ssa_debug_set_wait_limit_ns(100)
        try:
            all_calls(w)
            assert ssa.ssa_device_status(stream) in (ssa.SSA_OK, ssa.SSA_ERR_TIMEOUT)
            while ssa.ssa_device_status(stream) == ssa.SSA_ERR_TIMEOUT:  # one record per kernel
                pass
        finally:
            ssa.ssa_debug_set_wait_limit_ns(0)
        got = all_calls(w)
        torch.cuda.synchronize()
        ssa.device_status()
        for a, b in zip(want[w], got):
            assert torch.equal(a, b)
