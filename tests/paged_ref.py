"""Plain 64-bit forms of the paged-cache operators, and the bounds their results are held to.

Attention bound.  With u = 2^-24 and n visible keys, the fp32 score of a key is
off by at most ds = (D + 4) u S, S the largest scale * sum_d |q_d k_jd| of the
row (products, their sum in any order, and the product with the scale).  Every
weight is then off by a relative 2 ds (its own score and the maximum's) + 2^-21
(exponential) and the sum of n of them, kept through at most n steps, by n u.
The weights of 16-bit calls are rounded to the type (half a step, h) for the
product with the values.  So the row before its last rounding is off by at most
  (h + 2 (2 ds + 2^-21 + 2 n u)) V,   V = sum_j w_j |v_j| / sum_j w_j,
(numerator and denominator), and the output rounding adds h |out|.
"""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def attention(q, k, v, table, lens, starts, page, scale, causal=True, window=0):
    """(out, bound, lse, lse_bound) in float64, NaN in `out` for rows of no sequence."""
    q, k, v = q.cpu(), k.cpu(), v.cpu()
    dt = q.dtype
    T, hq, D = q.shape
    hk = k.shape[1]
    G = hq // hk
    B, width = table.shape
    starts = list(range(B + 1)) if starts is None else starts.tolist()
    out = torch.full((T, hq, D), math.nan, dtype=torch.float64)
    tol, lse, ltol = out.clone(), out[..., 0].clone(), out[..., 0].clone()
    u, h = 2.0 ** -24, HALF[dt]
    for b in range(B):
        a, e = starts[b], starts[b + 1]
        n = e - a
        L = max(0, min(int(lens[b]), width * page))
        j = torch.arange(L)
        pages = table[b].long()[j // page] if L else j
        ok = (pages >= 0) & (pages < k.shape[0] // page)
        slot = torch.where(ok, pages * page + j % page, torch.zeros_like(j))
        kk, vv = k[slot].double(), v[slot].double()
        for i in range(n):
            at = L - n + i
            see = ok.clone()
            if causal:
                see &= j <= at
                if window:
                    see &= at - j < window
            m = int(see.sum())
            if m == 0:
                out[a + i], tol[a + i] = 0.0, 0.0
                lse[a + i], ltol[a + i] = -math.inf, 0.0
                continue
            kx = kk[see].repeat_interleave(G, 1)
            vx = vv[see].repeat_interleave(G, 1)
            x = q[a + i].double()
            s = scale * (x[None] * kx).sum(-1)  # [m, hq]
            big = scale * (x[None] * kx).abs().sum(-1).amax(0)
            w = torch.softmax(s, 0)
            out[a + i] = (w[..., None] * vx).sum(0)
            V = (w[..., None] * vx.abs()).sum(0)
            ds = (D + 4) * u * big
            rel = (0.0 if dt == torch.float32 else h) + 2 * (2 * ds + 2.0 ** -21 + 2 * m * u)
            tol[a + i] = rel[:, None] * V
            lse[a + i] = torch.logsumexp(s, 0)
            ltol[a + i] = ds + 2.0 ** -21 + 2 * m * u + 8 * u * (lse[a + i].abs() + s.abs().amax(0))
    return out, tol, lse, ltol


def check_rows(got, out, tol, dt, inv_scale=None):
    """Rows of a sequence lie within the bound (the last rounding added)."""
    mine = ~torch.isnan(out[:, 0, 0])
    ref, t = out[mine], tol[mine]
    if inv_scale is None:
        g = got.cpu().double()[mine]
        t = t + HALF[dt] * (ref.abs() + t) + TINY[dt]
    else:
        g = got.cpu().view(torch.float8_e4m3fn).double()[mine]
        ref, t = (ref * inv_scale).clamp(-448, 448), t * inv_scale
        # half a step of E4M3: 2^-4 of the value, 2^-10 among the subnormals
        t = t + torch.maximum(2.0 ** -4 * (ref.abs() + t), torch.tensor(2.0 ** -10)) + 2.0 ** -23 * ref.abs()
    bad = ~((g - ref).abs() <= t)
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outside; worst "
                           f"{((g - ref).abs() / t).nan_to_num(1e9).max():.3g} of the bound; first {bad.nonzero()[:4].tolist()}")
