"""Workloads of the paged key/value cache and of sliding-window attention.

Each case is one pass through one operator as a program calls it: appending
rotated keys and values to a paged cache, sliding-window attention with sink
tokens over whole sequences (forward, or forward and backward), the attention
of single tokens over the paged cache, and the same for a batch whose
sequences share a long prefix.  ``run`` computes the operator in elementary
torch operations, or through the library where ``own`` is set; ``exact``
computes it in float64 from the definition.
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one new token for each of eight sequences: the cache write of a decode step
        {"name": "append_step", "op": "append", "dtype": "bf16", "B": 8, "Hq": 16, "Hkv": 4, "D": 128,
         "page": 64, "ctx": 8192, "tokens": 8, "ragged": False, "rot": 128, "interleaved": False},
        # sixteen prompts of mixed length packed into one buffer with rows to spare behind the last
        {"name": "append_prompts", "op": "append", "dtype": "bf16", "B": 16, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "ctx": 32768, "tokens": 16384, "ragged": True, "rot": 128, "interleaved": False},
        # float32, rotation of half the head in neighbouring pairs, odd lengths
        {"name": "append_f32", "op": "append", "dtype": "f32", "B": 5, "Hq": 4, "Hkv": 2, "D": 64,
         "page": 32, "ctx": 2000, "tokens": 777, "ragged": True, "rot": 32, "interleaved": True},
        # one short float32 sequence
        {"name": "window_f32", "op": "window", "dtype": "f32", "B": 1, "Hq": 2, "Hkv": 1, "T": 1000, "D": 64,
         "window": 256, "sinks": 4, "grad": False, "ragged": False, "rows": False},
        # prefill of a local layer at an 8k context, projections laid out token by token
        {"name": "window_prefill", "op": "window", "dtype": "bf16", "B": 1, "Hq": 16, "Hkv": 4, "T": 8192,
         "D": 128, "window": 1024, "sinks": 4, "grad": False, "ragged": False, "rows": True},
        # prefill of a local layer at a 64k context with a block of sink tokens
        {"name": "window_long", "op": "window", "dtype": "bf16", "B": 1, "Hq": 8, "Hkv": 8, "T": 65536,
         "D": 128, "window": 2048, "sinks": 64, "grad": False, "ragged": False, "rows": False},
        # training step in float32 on a padded batch of odd length
        {"name": "train_f32", "op": "window", "dtype": "f32", "B": 2, "Hq": 4, "Hkv": 2, "T": 777, "D": 64,
         "window": 128, "sinks": 4, "grad": True, "ragged": True, "rows": False},
        # training step of a local layer: the shape of the dual-stream training workload with shared heads
        {"name": "train", "op": "window", "dtype": "bf16", "B": 4, "Hq": 32, "Hkv": 8, "T": 4096, "D": 128,
         "window": 1024, "sinks": 4, "grad": True, "ragged": False, "rows": True},
        # one sequence, one token, a local layer deep into a 64k context: latency
        {"name": "decode_step", "op": "decode", "dtype": "bf16", "B": 1, "Hq": 16, "Hkv": 4, "D": 128,
         "page": 64, "ctx": 65536, "window": 1024, "sinks": 4},
        # a serving batch of mixed lengths, full attention over the cache: bandwidth
        {"name": "decode_batch", "op": "decode", "dtype": "bf16", "B": 32, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 64, "ctx": 32768, "window": 0, "sinks": 0},
        # eight answers to one prompt of 4k tokens
        {"name": "prefix_small", "op": "prefix", "dtype": "bf16", "B": 8, "Hq": 16, "Hkv": 4, "D": 128,
         "page": 64, "prefix": 4096, "ctx": 300},
        # sixty-four users behind one document of 32k tokens
        {"name": "prefix_large", "op": "prefix", "dtype": "bf16", "B": 64, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "prefix": 32768, "ctx": 1024},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "window", "window", "train", "decode", "prefix"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    c = {"op": op, "dtype": dtype, "D": D, "Hq": Hkv * rng.choice([1, 2, 3, 4, 8] if Hkv < 8 else [1, 2, 4]),
         "Hkv": Hkv}
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _log_int(rng, 1, 64)
        ragged = rng.random() < 0.6
        n = _log_int(rng, 1, 1024)
        return {**c, "B": B, "page": page, "ctx": _log_int(rng, 2 * n + 1, 8192),
                "tokens": min(16384, n * B) if ragged else B * min(n, 16384 // B), "ragged": ragged,
                "rot": rng.choice([D, D, D // 2, 24]), "interleaved": rng.random() < 0.5}
    if op in ("window", "train"):
        grad = op == "train"
        B = _log_int(rng, 1, 8)
        T = _log_int(rng, 16 if grad else 1, 16384)  # a token that sees itself alone has no gradient but rounding
        window = rng.choice([0, _log_int(rng, 8 if grad else 1, 2048), _log_int(rng, 16, 2048)])
        limit = (2e8 if grad else 4e8) / (16 if dtype == "f32" else 1)  # visible pairs
        while B * c["Hq"] * T * min(T, window or T) > limit:
            B, T = max(1, B // 2), T if B > 1 else T // 2 + 1
        return {**c, "op": "window", "B": B, "T": T, "window": window,
                "sinks": rng.choice([0, 1, 4, _log_int(rng, 1, 128)]) if window else 0, "grad": grad,
                "ragged": rng.random() < 0.4, "rows": rng.random() < 0.5}
    if op == "decode":
        B = _log_int(rng, 1, 64)
        window = rng.choice([0, 0, _log_int(rng, 1, 4096)])
        return {**c, "B": B, "page": page, "ctx": _log_int(rng, 1, min(65536, 262144 // B)), "window": window,
                "sinks": rng.choice([0, 4, _log_int(rng, 1, 128)]) if window else 0}
    B = _log_int(rng, 1, 64)
    return {**c, "B": B, "page": page, "prefix": _log_int(rng, 1, 32768), "ctx": _log_int(rng, 1, 1024)}


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)


def _lengths(gen, n, hi):
    """n lengths up to hi, the last of them hi."""
    x = torch.randint(0, hi + 1, (n,), generator=gen, device=DEV, dtype=torch.int32)
    x[-1] = hi
    return x


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 7919 + 17)
    dt, D, Hq, Hkv, B = _DT[case["dtype"]], case["D"], case["Hq"], case["Hkv"], case["B"]
    s = {"case": case, "scale": 1.0 / math.sqrt(D)}
    if case["op"] == "window":
        T = case["T"]

        def heads(H):
            if case["rows"]:  # [B, T, H, D] projections seen as [B, H, T, D]
                return _normal(gen, (B, T, H, D), dt).transpose(1, 2)
            return _normal(gen, (B, H, T, D), dt)

        s["q"], s["k"], s["v"] = heads(Hq), heads(Hkv), heads(Hkv)
        if case["grad"]:
            s["dh"] = heads(Hq)
        s["lens"] = _lengths(gen, B, T) if case["ragged"] else None
        return s
    page, ctx = case["page"], case["ctx"]
    per_seq = -(-ctx // page)
    shared = -(-case.get("prefix", 0) // page)
    n_pages = B * per_seq + shared + 1
    order = torch.randperm(n_pages, generator=gen, device=DEV).to(torch.int32)
    s["table"] = order[:B * per_seq].view(B, per_seq).contiguous()
    s["k_pages"] = _normal(gen, (n_pages, Hkv, page, D), dt)
    s["v_pages"] = _normal(gen, (n_pages, Hkv, page, D), dt)
    if case["op"] == "append":
        N = case["tokens"]
        s["q"], s["k"], s["v"] = _normal(gen, (N, Hq, D), dt), _normal(gen, (N, Hkv, D), dt), _normal(gen, (N, Hkv, D), dt)
        if case["ragged"]:  # N rows, a few of them (if there are many) behind the last sequence
            used = max(B, N - N // 50)
            cuts = torch.randint(0, used + 1, (B + 1,), generator=gen, device=DEV, dtype=torch.int32)
            cuts[0], cuts[-1] = 0, used
            s["q_start"] = cuts.sort().values.to(torch.int32)
            new = s["q_start"][1:] - s["q_start"][:-1]
            if (new > ctx).any():  # longer than the table holds: even shares instead
                s["q_start"] = (torch.arange(B + 1, device=DEV) * (min(used, B * ctx) // B)).to(torch.int32)
                new = s["q_start"][1:] - s["q_start"][:-1]
        else:
            s["q_start"] = None
            new = torch.full((B,), N // B, dtype=torch.int32, device=DEV)
        room = (ctx - new).double()
        s["lens"] = (torch.rand(B, generator=gen, device=DEV, dtype=torch.float64) * (room + 1)).floor().to(torch.int32)
        r = case["rot"]
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
        return s
    s["lens"] = _lengths(gen, B, ctx)
    s["q"] = _normal(gen, (B, Hq, D), dt)
    if shared:
        s["prefix_pages"] = order[B * per_seq:B * per_seq + shared].contiguous()
    return s


# ---------------------------------------------------------------- plain forms

def _softmax(x):
    """(weights, log-sum-exp) of the last axis; rows of -inf give zeros and -inf."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(x - m)
    l = e.sum(-1, keepdim=True)
    return e / torch.where(l > 0, l, torch.ones_like(l)), (m + torch.log(l)).squeeze(-1)


def _plain_window(s):
    c = s["case"]
    B, Hq, Hkv, T, D, W = c["B"], c["Hq"], c["Hkv"], c["T"], c["D"], c["window"] or c["T"]
    S = min(c["sinks"], T)
    n = min(max(W, 128), T)  # queries are cut into blocks of n: a block sees itself and the one before
    nb = -(-T // n)
    pad = nb * n - T

    def blocks(x, H):  # [B, H, T, D] -> [B, Hkv, H / Hkv, nb, n, D]
        return torch.nn.functional.pad(x.float(), (0, 0, 0, pad)).reshape(B, Hkv, H // Hkv, nb, n, D)

    def with_previous(x):
        if nb == 1:
            return x
        return torch.cat([torch.cat([torch.zeros_like(x[:, :, :, :1]), x[:, :, :, :-1]], 3), x], 4)

    q, kb, vb = blocks(s["q"], Hq), blocks(s["k"], Hkv), blocks(s["v"], Hkv)
    first_k, first_v = kb.reshape(B, Hkv, 1, 1, nb * n, D)[..., :S, :], vb.reshape(B, Hkv, 1, 1, nb * n, D)[..., :S, :]
    k2, v2 = with_previous(kb), with_previous(vb)
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device=DEV)
    lens = lens.view(B, 1, 1, 1, 1, 1)
    t = torch.arange(nb * n, device=DEV).view(nb, n, 1)
    key = torch.arange(nb, device=DEV).view(nb, 1, 1) * n + torch.arange(k2.shape[4], device=DEV) - (n if nb > 1 else 0)
    near = (key <= t) & (key > t - W) & (key >= 0)
    sink = (torch.arange(S, device=DEV) <= t - W)  # the sinks that the window has left behind
    seen = torch.cat([sink, near], -1) & (t < lens)
    x = torch.cat([q @ first_k.transpose(-1, -2), q @ k2.transpose(-1, -2)], -1) * s["scale"]
    p, lse = _softmax(x.masked_fill(~seen, float("-inf")))
    h = p[..., :S] @ first_v + p[..., S:] @ v2

    def whole(x, like):  # [B, Hkv, g, nb, n, D] -> [B, H, T, D]
        return x.reshape(B, -1, nb * n, D)[:, :, :T].to(like.dtype)

    out = {"h": whole(h, s["q"]), "lse": lse.reshape(B, Hq, nb * n)[:, :, :T].contiguous()}
    if c["grad"]:
        dh = blocks(s["dh"], Hq)
        dp = torch.cat([dh @ first_v.transpose(-1, -2), dh @ v2.transpose(-1, -2)], -1)
        ds = p * (dp - (dp * p).sum(-1, keepdim=True)) * s["scale"]
        out["dq"] = whole(ds[..., :S] @ first_k + ds[..., S:] @ k2, s["q"])

        def to_keys(w, x):  # sum over queries and over the heads of a group, back at the keys' places
            near = (w[..., S:].transpose(-1, -2) @ x).sum(2)
            if nb > 1:
                own_block, before = near[..., n:, :], near[..., :n, :]
                near = own_block + torch.cat([before[:, :, 1:], torch.zeros_like(before[:, :, :1])], 2)
            near = near.reshape(B, Hkv, nb * n, D)
            near[:, :, :S] += (w[..., :S].transpose(-1, -2) @ x).sum((2, 3))
            return near[:, :, :T].to(s["k"].dtype)

        out["dk"], out["dv"] = to_keys(ds, q), to_keys(p, dh)
    return out


def _rotate(x, pos, inv_freq, interleaved):
    """Rotation of x [N, H, D] (float32) by pos [N] (float64): pairs (i, i + r/2), or neighbours."""
    r = 2 * inv_freq.numel()
    angle = pos[:, None, None].double() * inv_freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_append(s):
    c = s["case"]
    N, B, page = c["tokens"], c["B"], c["page"]
    i = torch.arange(N, device=DEV)
    start = s["q_start"].long() if s["q_start"] is not None else torch.arange(B + 1, device=DEV) * (N // B)
    b = torch.searchsorted(start, i, right=True) - 1
    real = b < B  # rows behind the last sequence belong to none
    b = b.clamp(max=B - 1)
    pos = s["lens"].long()[b] + i - start[b]
    width = s["table"].shape[1]
    pages = s["table"].long()[b, (pos // page).clamp(max=width - 1)]
    q = torch.where(real[:, None, None], _rotate(s["q"].float(), pos, s["inv_freq"], c["interleaved"]).to(s["q"].dtype), s["q"])
    k = _rotate(s["k"].float(), pos, s["inv_freq"], c["interleaved"]).to(s["k"].dtype)
    at = pages * page + pos % page
    # rows behind the last sequence write what the first token writes, where it does
    slot, token = torch.where(real, at, at[0]), torch.where(real, i, torch.zeros_like(i))
    s["k_pages"][slot // page, :, slot % page] = k[token]
    s["v_pages"][slot // page, :, slot % page] = s["v"][token]
    lens = s["lens"] + (start[1:] - start[:-1]).to(torch.int32)
    return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"], "lens": lens}


def _tokens(pages, at, page):
    """The tokens at `at` (slots of the pool) of the pages [n, Hkv, page, D] -> [..., Hkv, D] in float32."""
    return pages[at // page, :, at % page].float()


def _of_table(s):
    """(keys, values, which of them count) of each sequence: [B, L, Hkv, D] and [B, L]."""
    c = s["case"]
    page, ctx, S = c["page"], c["ctx"], c.get("sinks", 0)
    W = min(c.get("window", 0) or ctx, ctx)
    lens = s["lens"].long()[:, None]
    near = lens - W + torch.arange(W, device=DEV) if W < ctx else torch.arange(ctx, device=DEV).expand(c["B"], ctx)
    first = torch.arange(S, device=DEV).expand(c["B"], S)
    pos = torch.cat([first, near], 1)
    seen = torch.cat([first < lens, (near >= S) & (near < lens) & (near >= lens - W)], 1)
    pos = pos.clamp(0, ctx - 1)
    at = torch.gather(s["table"].long(), 1, pos // page) * page + pos % page
    return _tokens(s["k_pages"], at, page), _tokens(s["v_pages"], at, page), seen


def _plain_decode(s):
    c = s["case"]
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    k, v, seen = _of_table(s)
    q = s["q"].float().view(B, Hkv, -1, D)
    x = q @ k.permute(0, 2, 3, 1) * s["scale"]
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    v = v.permute(0, 2, 1, 3)
    if c["op"] == "decode":
        p, lse = _softmax(x)
        h = p @ v
    else:
        P = torch.arange(c["prefix"], device=DEV)
        at = s["prefix_pages"].long()[P // c["page"]] * c["page"] + P % c["page"]
        kp, vp = _tokens(s["k_pages"], at, c["page"]).transpose(0, 1), _tokens(s["v_pages"], at, c["page"]).transpose(0, 1)
        rows = q.transpose(0, 1).reshape(Hkv, -1, D)  # the whole batch against the prefix at once
        y = (rows @ kp.transpose(-1, -2) * s["scale"]).view(Hkv, B, -1, c["prefix"]).transpose(0, 1)
        p, lse = _softmax(torch.cat([y, x], -1))
        of_prefix = p[..., :c["prefix"]].transpose(0, 1).reshape(Hkv, -1, c["prefix"]) @ vp
        h = of_prefix.view(Hkv, B, -1, D).transpose(0, 1) + p[..., c["prefix"]:] @ v
    return {"h": h.reshape(B, c["Hq"], D).to(s["q"].dtype), "lse": lse.reshape(B, c["Hq"])}


def _library(s):
    from block_sparse_full_b200 import ssa

    c = s["case"]
    if c["op"] == "window":
        p = ssa.window_params_for(s["q"], s["k"], c["window"], c["sinks"], s["scale"])
        out = ssa.window_fwd(p, s["q"], s["k"], s["v"], lens=s["lens"])
        if not c["grad"]:
            return out
        dq, dk, dv = ssa.window_bwd(p, s["q"], s["k"], s["v"], out, s["dh"], lens=s["lens"])
        return {**out, "dq": dq, "dk": dk, "dv": dv}
    p = ssa.cache_params_for(s["q"], s["k_pages"], s["table"], c.get("window", 0), c.get("sinks", 0), s["scale"])
    if c["op"] == "append":
        out = ssa.cache_append(p, s["k_pages"], s["v_pages"], s["table"], s["lens"], s["k"], s["v"], q=s["q"],
                               inv_freq=s["inv_freq"], interleaved=c["interleaved"], q_start=s["q_start"])
        return {"q": out["q"], "k_pages": s["k_pages"], "v_pages": s["v_pages"], "lens": out["lens"]}
    if c["op"] == "decode":
        return ssa.paged_decode(p, s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"])
    return ssa.prefix_decode(p, s["q"], s["k_pages"], s["v_pages"], s["prefix_pages"], c["prefix"], s["table"],
                             s["lens"])


def run(state):
    if own:
        return _library(state)
    if state["case"]["op"] == "window":
        return _plain_window(state)
    if state["case"]["op"] == "append":
        return _plain_append(state)
    return _plain_decode(state)


# ---------------------------------------------------------------- what a pass needs at least

def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "window":
        T = case["T"]
        W = min(case["window"] or T, T)
        # visible (query, key) pairs of one head; half of a padded batch is padding on average
        pairs = W * (W + 1) / 2 + (T - W) * W + sum(max(0, T - W - j) for j in range(min(case["sinks"], T)))
        share = 0.5 * (1 + 1 / B) if case["ragged"] else 1.0
        flops = 4.0 * B * Hq * pairs * D * share
        nbytes = B * T * D * esz * (2 * Hq + 2 * Hkv) + 4.0 * B * Hq * T
        if case["grad"]:
            flops *= 3.5  # five more products
            nbytes += B * T * D * esz * (2 * Hq + 2 * Hkv)
        return {"bytes": nbytes, "flops": flops}
    if case["op"] == "append":
        n = case["tokens"] - (case["tokens"] // 50 if case["ragged"] else 0)
        return {"bytes": 2.0 * n * D * esz * (Hq + 2 * Hkv), "flops": 3.0 * n * (Hq + Hkv) * case["rot"]}
    mean = 0.5 * case["ctx"] * (1 + 1 / B)  # lengths are spread evenly, the last is the longest
    if case.get("window", 0):
        mean = min(mean, case["window"] + case["sinks"])
    keys = B * mean + case.get("prefix", 0)
    pairs = B * (mean + case.get("prefix", 0))
    return {"bytes": 2.0 * keys * Hkv * D * esz + 2.0 * B * Hq * D * esz + 4.0 * B * Hq, "flops": 4.0 * pairs * Hq * D}


# ---------------------------------------------------------------- definitions in 64 bits

def _attend(q, k, v, keep, scale):
    """softmax(scale q k^T over keep) v -> (h, weights, log-sum-exp), float64; rows without a key give 0 and -inf."""
    x = (q @ k.T * scale).masked_fill(~keep, -math.inf)
    lse = torch.logsumexp(x, -1)
    w = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    return w @ v, w, lse


def _exact_window(s):
    c = s["case"]
    B, Hq, T, D = s["q"].shape
    G, W = Hq // c["Hkv"], c["window"] or T
    f64 = dict(dtype=torch.float64, device=DEV)
    out = {"h": torch.zeros(B, Hq, T, D, **f64), "lse": torch.full((B, Hq, T), -math.inf, **f64)}
    if c["grad"]:
        out.update(dq=torch.zeros(B, Hq, T, D, **f64), dk=torch.zeros(B, c["Hkv"], T, D, **f64),
                   dv=torch.zeros(B, c["Hkv"], T, D, **f64))
    for b in range(B):
        n = int(s["lens"][b]) if s["lens"] is not None else T
        for h in range(Hq):
            q, k, v = s["q"][b, h].double(), s["k"][b, h // G].double(), s["v"][b, h // G].double()
            for t0 in range(0, n, 2048):
                t1 = min(n, t0 + 2048)
                t, j = torch.arange(t0, t1, device=DEV)[:, None], torch.arange(t1, device=DEV)
                keep = (j <= t) & ((j > t - W) | (j < c["sinks"]))
                o, w, lse = _attend(q[t0:t1], k[:t1], v[:t1], keep, s["scale"])
                out["h"][b, h, t0:t1], out["lse"][b, h, t0:t1] = o, lse
                if c["grad"]:
                    g = s["dh"][b, h, t0:t1].double()
                    dx = w * (g @ v[:t1].T - (g * o).sum(-1, keepdim=True)) * s["scale"]
                    out["dq"][b, h, t0:t1] = dx @ k[:t1]
                    out["dk"][b, h // G, :t1] += dx.T @ q[t0:t1]
                    out["dv"][b, h // G, :t1] += w.T @ g
    return out


def _exact_rotation(x, pos, inv_freq, interleaved):
    y = x.double().clone()
    for i in range(inv_freq.numel()):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + inv_freq.numel())
        z = torch.complex(y[..., a], y[..., b]) * torch.exp(1j * pos * inv_freq[i])[:, None]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_append(s):
    c = s["case"]
    N, B, page = c["tokens"], c["B"], c["page"]
    cuts = s["q_start"].tolist() if s["q_start"] is not None else [b * (N // B) for b in range(B + 1)]
    out = {"q": s["q"].double().clone(), "k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double(),
           "lens": s["lens"].clone()}
    for b in range(B):
        i0, i1 = cuts[b], cuts[b + 1]
        pos = int(s["lens"][b]) + torch.arange(i1 - i0, device=DEV, dtype=torch.int64)
        where = s["table"][b].long()[pos // page]
        turn = (pos.double(), s["inv_freq"], c["interleaved"])
        out["q"][i0:i1] = _exact_rotation(s["q"][i0:i1], *turn)
        out["k_pages"][where, :, pos % page] = _exact_rotation(s["k"][i0:i1], *turn)
        out["v_pages"][where, :, pos % page] = s["v"][i0:i1].double()
        out["lens"][b] += i1 - i0
    return out


def _exact_decode(s):
    c = s["case"]
    B, Hq, D = s["q"].shape
    G, page = Hq // c["Hkv"], c["page"]
    out = {"h": torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV),
           "lse": torch.zeros(B, Hq, dtype=torch.float64, device=DEV)}

    def dense(pages, ids, n):  # the first n tokens of the pages `ids`: [Hkv, n, D]
        return pages[ids.long()].double().transpose(0, 1).reshape(c["Hkv"], -1, D)[:, :n]

    P = c.get("prefix", 0)
    for b in range(B):
        n = int(s["lens"][b])
        used = s["table"][b, :-(-n // page)]
        k, v = dense(s["k_pages"], used, n), dense(s["v_pages"], used, n)
        keep = torch.ones(1, P + n, dtype=torch.bool, device=DEV)
        if P:
            k = torch.cat([dense(s["k_pages"], s["prefix_pages"], P), k], 1)
            v = torch.cat([dense(s["v_pages"], s["prefix_pages"], P), v], 1)
        elif c["window"]:
            j = torch.arange(n, device=DEV)
            keep = ((j >= n - c["window"]) | (j < c["sinks"]))[None]
        for h in range(Hq):
            o, _, lse = _attend(s["q"][b, h:h + 1].double(), k[h // G], v[h // G], keep, s["scale"])
            out["h"][b, h], out["lse"][b, h] = o[0], lse[0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "window":
        return _exact_window(s)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_decode(s)
