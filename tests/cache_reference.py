"""64-bit references of the cache-append, windowed and block-scaled decode
operators on the CPU, written token by token, with the bounds that the
kernels' roundings allow.

Units of rounding (half a step): bf16 2^-8, f16 2^-11, fp32 2^-24, e4m3 2^-4
relative; below the smallest normal number half the subnormal step.
"""
from __future__ import annotations

import math

import torch

Q_MAX = {"fp8_e4m3_block": 448.0, "int8_block": 127.0, "fp8_e4m3_pth": 448.0, "int8_pth": 127.0, "int4_pth": 7.0}


# ------------------------------------------------------------------ decode

def window_decode(q, k, v, n, scale, window, sinks, *, code_v=None, s_v=None, half_p=False):
    """One request.  q [L, Hq, D], k and v [n, Hkv, D] (float64, values); code_v, s_v: V as codes and per-token
    scales where it is held in 8 bits.  Returns out [L, Hq, D], lse [L, Hq] and their error bounds.

    The bounds: the logits are fp32 sums of exact products, off by ex = 2^-21 sum|q k| scale (a sum of up to 128
    terms in any order, twice over) + the bf16 -> f16 conversion's 2^-25 per subnormal entry; the base-2
    exponentials and the sums over n keys and up to n partials add 2^-20 + n 2^-24; P is rounded to bf16 (2^-8) or
    f16 (2^-11, or 2^-25 of the largest weight where it is subnormal); the output to bf16 (2^-8)."""
    L, Hq, D = q.shape
    Hkv = k.shape[1] if k.numel() else 1
    grp = Hq // max(1, Hkv)
    out = torch.zeros(L, Hq, D, dtype=torch.float64)
    lse = torch.full((L, Hq), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for i in range(L):
        p = n - L + i
        if p < 0:
            continue
        t = torch.arange(p + 1)
        t = t[(t < sinks) | (t > p - window)]
        for h in range(Hq):
            kk, vv = k[t, h // grp], v[t, h // grp]
            x = kk @ q[i, h] * scale
            w = torch.exp(x - x.max())
            total = w.sum()
            out[i, h] = (w @ vv) / total
            lse[i, h] = x.max() + math.log(float(total))
            ex = float((kk.abs() @ q[i, h].abs()).max()) * abs(scale) * 2 ** -21
            ex += 2 ** -20 + len(t) * 2 ** -24
            weight = (w @ vv.abs()) / total
            if half_p:
                ex += D * 2 ** -25 * float(kk.abs().max()) * abs(scale)
                ws = w * s_v[t, h // grp] if s_v is not None else w
                codes = code_v[t, h // grp] if code_v is not None else vv
                extra = weight * 2 ** -11 + 2 ** -25 * float(ws.max()) * codes.abs().sum(0) / total
            else:
                extra = weight * 2 ** -8
            tol_o[i, h] = extra + 4 * ex * weight + out[i, h].abs() * 2 ** -8 + 1e-30
            tol_l[i, h] = 2 * ex + 2 ** -22 * abs(float(lse[i, h]))
    return out, lse, tol_o, tol_l


def gather(cache, block_table, b, n, page, plane):
    """Rows of tokens 0 .. n - 1 of request b; a token whose page has no valid block id gives zeros."""
    rows = torch.zeros((n,) + cache.shape[3:], dtype=torch.float64)
    for j in range(-(-n // page)):
        blk = int(block_table[b, j])
        m = min(page, n - j * page)
        if 0 <= blk < cache.shape[0]:
            rows[j * page:j * page + m] = cache[blk, plane, :m].double()
    return rows


def token_scales(scales, block_table, b, n, page, plane):
    """Per-token scales [n, Hkv] of request b."""
    G = page // scales.shape[2]
    out = torch.zeros(n, scales.shape[3], dtype=torch.float64)
    for t in range(n):
        blk = int(block_table[b, t // page])
        if 0 <= blk < scales.shape[0]:
            out[t] = scales[blk, plane, t % page // G].double()
    return out


# ------------------------------------------------------------------ append

def rotate(x, row, interleaved):
    """x [heads, D] float64 at the angles of one table row; returns (rotated, |x| + |y| of each column's pair)."""
    r = row.numel()
    y, mag = x.clone(), x.abs()
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        c, s = float(row[i]), float(row[r // 2 + i])
        y[:, a] = x[:, a] * c - x[:, b] * s
        y[:, b] = x[:, b] * c + x[:, a] * s
        mag[:, a] = mag[:, b] = x[:, a].abs() + x[:, b].abs()
    return y, mag


def grid_e4m3(y):
    y = y.clamp(-448.0, 448.0)
    e = torch.frexp(y.abs())[1].double() - 1.0
    step = torch.exp2(e.clamp(min=-6.0) - 3.0)
    return torch.round(y / step) * step


def grid_int(y, top):
    return torch.round(y).clamp(-top, top)


def grid(y, kv):
    if kv.startswith("fp8"):
        return grid_e4m3(y)
    return grid_int(y, Q_MAX[kv])


def code_range(y, off, kv):
    """The smallest and largest code that a value within y +- off may round to."""
    return grid(y - off, kv), grid(y + off, kv)
