"""64-bit references of the attention-side operators, on the CPU, from their definitions, and the
bounds that the GPU results are held to.  A rounding to a type t is off by at most eps(t)/2."""
from __future__ import annotations

import math

import torch

HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
E4M3_HALF = 2.0 ** -4


def norm_ref(x, res, w, eps):
    """(r, n) in 64 bits."""
    r = x.double().cpu() + (res.double().cpu() if res is not None else 0.0)
    n = r / torch.sqrt(r.square().mean(-1, keepdim=True) + eps)
    return r, n * w.double().cpu() if w is not None else n


def rope_ref(x, positions, inv_freq, rot, style):
    """(rotated x, |a| + |b| of each element's pair) in 64 bits; x [T][H][D]."""
    x = x.double().cpu().clone()
    mag = torch.zeros_like(x)
    angle = positions.double().cpu()[:, None] * inv_freq.cpu()[None, :]
    for i in range(rot // 2):
        ia, ib = (i, i + rot // 2) if style == 0 else (2 * i, 2 * i + 1)
        a, b = x[:, :, ia].clone(), x[:, :, ib].clone()
        c, s = torch.cos(angle[:, i])[:, None], torch.sin(angle[:, i])[:, None]
        x[:, :, ia], x[:, :, ib] = a * c - b * s, b * c + a * s
        mag[:, :, ia] = mag[:, :, ib] = a.abs() + b.abs()
    return x, mag


def attn_ref(q, keys, values, scale, visible):
    """One KV head's rows: q [R][D], keys/values [N][D], visible bool [R][N].  Returns
    (out, lse, tolerance of out, tolerance of lse) in 64 bits; masked keys never enter a product.

    Tolerances: fp32 scores are off by e = 2 D 2^-24 max sum|q k| scale (products are exact; the
    factor 2 for sums that truncate), so probabilities by 2 e relatively; the probabilities'
    rounding to 16 bits by eps/2; fp32 exponentials and sums by 2^-18; fp16 probabilities below
    2^-14 by 2^-25 each; the output's own rounding by eps/2."""
    t = q.dtype
    q, keys, values = q.double(), keys.double(), values.double()
    R, D = q.shape
    out = torch.zeros(R, D, dtype=torch.float64)
    lse = torch.full((R,), -math.inf, dtype=torch.float64)
    tol = torch.zeros(R, D, dtype=torch.float64)
    tol_lse = torch.zeros(R, dtype=torch.float64)
    for r in range(R):
        idx = visible[r].nonzero().flatten()
        if idx.numel() == 0:
            continue
        k, v = keys[idx], values[idx]
        s = (k @ q[r]) * scale
        lse[r] = torch.logsumexp(s, 0)
        p = torch.exp(s - lse[r])
        out[r] = p @ v
        e = 2 * D * 2.0 ** -24 * float((k.abs() @ q[r].abs()).max()) * scale
        tol[r] = HALF[t] * out[r].abs() + (HALF[t] + 2 * e + 2.0 ** -18) * (p @ v.abs())
        if t == torch.float16:
            tol[r] += idx.numel() * 2.0 ** -25 * v.abs().max() + 2.0 ** -25
        tol_lse[r] = e + 2.0 ** -20 * (1 + abs(float(lse[r])))
    return out, lse, tol, tol_lse
