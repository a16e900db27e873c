"""Float64 references of window attention, the paged cache and its attention,
with elementwise error bounds of the kernels' arithmetic.

The bounds count, to first order, with u(t) = torch.finfo(t).eps / 2:
  scores   an inner product of D terms in float32 and its scaling are off by at
           most (D + 8) u(f32) sum|q||k| sm_scale; float32 accumulation on the
           tensor cores may truncate, so that u is doubled (e_x);
  weights  2^x instructions and the exponent's rounding: 2^-18 (w);
  bf16     weights (and score gradients) are rounded to bf16 before their
           product with values, keys or queries: u(bf16) each (r);
  outputs  rounded once: u(dtype) (o).
An output sum_s p_s v_s with weights off by a relative e is off by at most
2 e sum_s p_s |v_s| (2: numerator and normaliser).
"""
import math

import torch

U32 = torch.finfo(torch.float32).eps / 2
W = 2.0 ** -18


def u(dtype):
    return torch.finfo(dtype).eps / 2


def keep_mask(T, window, sinks, length):
    t = torch.arange(T)[:, None]
    s = torch.arange(T)[None, :]
    near = s <= t if window == 0 else (s <= t) & ((s > t - window) | (s < sinks))
    return near & (t < length)


def attend(q, k, v, keep, scale, dtype):
    """One head, float64: dict(h, lse, p, and the bounds h_tol, lse_tol, w_tol)."""
    D = q.shape[-1]
    x = (q @ k.T) * scale
    x = torch.where(keep, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1) if x.shape[-1] else torch.full(x.shape[:1], -math.inf, dtype=torch.float64)
    some = torch.isfinite(lse)
    p = torch.where(keep, torch.exp(x - torch.where(some, lse, torch.zeros_like(lse))[:, None]), torch.zeros_like(x))
    h = p @ v
    size = torch.where(keep, (q.abs() @ k.abs().T) * scale, torch.zeros_like(x))
    top = size.amax(-1) if x.shape[-1] else torch.zeros(x.shape[:1], dtype=torch.float64)
    e_x = 2 * (D + 8) * U32 * top + W + 4 * U32 * torch.where(some, lse.abs(), torch.zeros_like(lse))
    r = u(dtype) if dtype == torch.bfloat16 else 0.0
    h_tol = (2 * e_x[:, None] + r + 64 * U32) * (p @ v.abs()) + u(dtype) * h.abs()
    return {"h": h, "lse": lse, "p": p, "h_tol": h_tol, "lse_tol": 2 * e_x, "w_tol": 2 * e_x}


def window(q, k, v, W_, S, lens, scale, dh=None):
    """[B,H,T,D] tensors -> dict of float64 results and bounds ("<name>_tol")."""
    dtype = q.dtype
    q, k, v = q.double(), k.double(), v.double()
    B, Hq, T, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    out = {"h": z(B, Hq, T, D), "h_tol": z(B, Hq, T, D), "lse": z(B, Hq, T), "lse_tol": z(B, Hq, T)}
    if dh is not None:
        dh = dh.double()
        for n, like in (("dq", q), ("dk", k), ("dv", v)):
            out[n], out[n + "_tol"] = torch.zeros_like(like), torch.zeros_like(like)
    r = u(dtype) if dtype == torch.bfloat16 else 0.0
    for b in range(B):
        n = T if lens is None else int(lens[b])
        keep = keep_mask(T, W_, S, n)
        rows, cols = torch.arange(T) < n, torch.arange(T) < n
        for h in range(Hq):
            clean = lambda x: torch.where(rows[:, None], x, torch.zeros_like(x))  # noqa: E731
            qq, kk, vv = clean(q[b, h]), clean(k[b, h // G]), clean(v[b, h // G])
            a = attend(qq, kk, vv, keep, scale, dtype)
            for name in ("h", "h_tol", "lse", "lse_tol"):
                out[name][b, h] = a[name]
            if dh is None:
                continue
            g, p, w = clean(dh[b, h]), a["p"], a["w_tol"][:, None]
            dp = g @ vv.T
            delta = (g * a["h"]).sum(-1, keepdim=True)
            ds = p * (dp - delta) * scale
            e_dp = 2 * (D + 8) * U32 * (g.abs() @ vv.abs().T)
            e_delta = (g.abs() * (a["h_tol"] + (D + 8) * U32 * a["h"].abs())).sum(-1, keepdim=True)
            ds_tol = (w + r + 8 * U32) * ds.abs() + p * (e_dp + e_delta) * scale
            p_tol = (w + r + 8 * U32) * p
            acc = 2 * (T + 8) * U32 * 0.1  # sums over T tokens: their roundings are independent
            out["dq"][b, h] = ds @ kk
            out["dq_tol"][b, h] = ds_tol @ kk.abs() + acc * (ds.abs() @ kk.abs())
            out["dk"][b, h // G] += ds.T @ qq
            out["dk_tol"][b, h // G] += ds_tol.T @ qq.abs() + acc * (ds.abs().T @ qq.abs())
            out["dv"][b, h // G] += p.T @ g
            out["dv_tol"][b, h // G] += p_tol.T @ g.abs() + acc * (p.T @ g.abs())
    if dh is not None:
        for n in ("dq", "dk", "dv"):
            out[n + "_tol"] += u(dtype) * out[n].abs()
    return out


def check(got, ref, names, tiny=1e-30):
    """Every element within its bound; infinities equal."""
    for n in names:
        x, y, tol = got[n].detach().double().cpu(), ref[n], ref[n + "_tol"]
        assert x.shape == y.shape, (n, x.shape, y.shape)
        fine = torch.isfinite(y)
        assert torch.equal(x[~fine], y[~fine]), f"{n}: infinities differ"
        assert torch.isfinite(x[fine]).all(), f"{n}: not finite"
        d = (x - y).abs()[fine]
        over = d - tol[fine] - tiny
        assert (over <= 0).all(), (f"{n}: off by {d.max().item():.3e}, worst {(d / (tol[fine] + tiny)).max().item():.2f} "
                                   f"times its bound at {int((over > 0).sum())} of {d.numel()}")


def rotate(x, pos, inv_freq, interleaved):
    """x [N,H,D] float64 rotated to pos [N]."""
    y = x.clone()
    n = 0 if inv_freq is None else inv_freq.numel()
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        c, s = torch.cos(pos.double() * inv_freq[i])[:, None], torch.sin(pos.double() * inv_freq[i])[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def rotate_tol(x, dtype):
    """Bound of the kernel's rotation: the angle's float32 form and the sines (2^-21 of a pair's
    size together), two products and their rounding, and the output's rounding."""
    return (2.0 ** -20 + u(dtype)) * x.double().abs().amax(-1, keepdim=True) * 2
