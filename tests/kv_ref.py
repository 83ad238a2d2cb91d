"""Plain float64 forms of the paged cache's operators (test infrastructure), and
how far float32 arithmetic in any order may be from them."""
import math

import torch

from tests.serving_ref import HALF, TINY

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def quantise(rows, quant, static=None):
    """16-bit rows [..., D] -> (E4M3 codes as uint8, scales [...] or None), every step one IEEE float32 operation: the
    bits are determined."""
    x = rows.float()
    if quant == "row":
        c = torch.clamp(torch.nan_to_num(x.abs(), nan=0.0, posinf=math.inf).amax(-1) / F8_MAX, min=2.0 ** -100)
        c1 = c[..., None]
        y = torch.where(c1 > 2.0 ** 100, x * (1.0 / c1), x / c1)
    else:
        c, y = None, x / torch.tensor(static, dtype=torch.float32)
    y = torch.where(y > F8_MAX, F8_MAX, torch.where(y < -F8_MAX, -F8_MAX, y))
    return y.to(F8).view(torch.uint8), c


def rows_of(cache, page, slot):
    """float64 (k, v) rows [n, kv_heads, D] of a cache (k, v, k_scale, v_scale) on the host."""
    got = []
    for t, c in ((cache[0], cache[2]), (cache[1], cache[3])):
        if t.dtype in (torch.uint8, F8):
            r = t.view(torch.uint8)[page, :, slot].view(F8).float().double()
            got.append(r * (c[page, :, slot].double()[..., None] if isinstance(c, torch.Tensor)
                            else float(torch.tensor(c, dtype=torch.float32))))
        else:
            got.append(t[page, :, slot].double())
    return got


def attention(q, cache, table, lengths, scale, window):
    """q [B, heads, D], all on the host -> float64 (out, lse, out's tolerance before its rounding, lse's tolerance).

    The tolerance: a score of D products summed in float32 in any order is off by at most (D + 8) 2^-24 of
    scale * sum |q k| (twice that allowed: the matrix unit's additions are not rounded to nearest), its exponent by 2^-23 of the largest score
    besides, and exp2 by 2^-22: rho in all, so the quotient by 2 rho; n additions to the sums by n 2^-23; the
    weights' two parts by 2^-16 each (bf16, E4M3 values), fp16's by no less than 2^-25 of a sum that is 1 or more."""
    B, heads, D = q.shape
    P, H = cache[0].shape[2], cache[0].shape[1]
    pages = cache[0].shape[0]
    G = heads // H
    out, tol = torch.zeros((B, heads, D), dtype=torch.float64), torch.zeros((B, heads, D), dtype=torch.float64)
    lse, ltol = torch.full((B, heads), -math.inf, dtype=torch.float64), torch.zeros((B, heads), dtype=torch.float64)
    for b in range(B):
        n = min(max(int(lengths[b]), 0), table.shape[1] * P)
        t = torch.arange(max(0, n - window) if window else 0, n)
        page = table[b].long()[t // P]
        t, page = t[(page >= 0) & (page < pages)], page[(page >= 0) & (page < pages)]
        if not len(t):
            continue
        k, v = rows_of(cache, page, t % P)
        for h in range(heads):
            kh, vh, qh = k[:, h // G], v[:, h // G], q[b, h].double()
            s = (kh @ qh) * scale
            p = torch.exp(s - s.max())
            lse[b, h] = s.max() + torch.log(p.sum())
            out[b, h] = (p[:, None] * vh).sum(0) / p.sum()
            rho = float(((kh.abs() @ qh.abs()) * abs(scale)).max()) * (D + 8) * 2.0 ** -23 \
                + float(s.abs().max()) * 2.0 ** -22 + 2.0 ** -22
            share = (p[:, None] * vh.abs()).sum(0) / p.sum()
            tol[b, h] = share * (2 * rho + (len(t) + 64) * 2.0 ** -23 + 2.0 ** -16) \
                + len(t) * 2.0 ** -25 * float(vh.abs().max())
            ltol[b, h] = rho + (len(t) + 64) * 2.0 ** -23 + 2.0 ** -22 * abs(float(lse[b, h]))
    return out, lse, tol, ltol


def assert_near(got, want, tol, act):
    """got of the 16-bit type against float64 with its tolerance and one rounding."""
    got = got.cpu().double()
    both = torch.isnan(got) & torch.isnan(want)
    off = (got - want).abs() - tol
    bad = ~((off <= HALF[act] * (want.abs() + tol) + TINY[act]) | both)
    assert not bool(bad.any()), (int(bad.sum()), float(off[bad].max()), bad.nonzero()[:4].tolist())
