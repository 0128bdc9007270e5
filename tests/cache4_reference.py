"""The 4-bit cache in plain torch: the quantiser's formula, attention to the stored
values in 64 bits with bounds for the kernel, and eviction by accumulated weight.

Bounds (u = 2^-8, half a bf16 step): a score is a sum of 32-element products of the
query with 16 + code (at most 31), in fp32, times the scale, plus the minimum's term:
  e_s = scale (D + 16) 2^-23 sum_d |q_d| (31 c_g + |m_g|), the largest of the keys
  O   : u |O| + (u + 2 e_s + n 2^-23) sum_j p |v - mid| + (2 e_s + n 2^-23) sum_j p |mid|
        with mid = m + 8 c: only p c (code - 8) passes through bf16
  lse : e_s + 2^-20 (1 + |lse|)
  w   : (2.1 e_s + 2^-19) p + 2^-23 |w|
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8


def quantise(x):
    """bf16 [..., D] -> fp32 (codes, minima, scales), groups of 32 elements, rounding as
    the formula has it in fp32."""
    g = x.float().unflatten(-1, (-1, 32))
    mn = g.amin(-1)
    c = ((g.amax(-1) - mn) / 15).to(torch.bfloat16).float()
    z = ((g - mn[..., None]) / torch.where(c > 0, c, torch.ones_like(c))[..., None]).round()
    z = torch.where(c[..., None] > 0, z.clamp(0, 15), torch.zeros_like(z))
    return z, mn, c


def stored(x):
    """fp64 (values, mid, largest code term 31 c + |m|) a cache holds for x [..., D]."""
    z, mn, c = (t.double() for t in quantise(x))
    v = mn[..., None] + c[..., None] * z
    mid = (mn + 8 * c)[..., None].expand_as(v)
    big = (31 * c + mn.abs())[..., None].expand_as(v)
    return tuple(t.flatten(-2) for t in (v, mid, big))


def attend(q, k, v, scale=None):
    """q bf16 [Hq, D], k, v bf16 [n, Hkv, D] as appended -> dict of fp64 results and
    bounds: o [Hq, D], lse [Hq], p [Hkv, n] summed over the group."""
    Hq, D = q.shape
    n, Hkv, _ = k.shape
    scale = 1 / math.sqrt(D) if scale is None else scale
    if n == 0:
        z = torch.zeros(Hq, D, dtype=torch.float64)
        return dict(o=z, o_tol=z, lse=torch.full((Hq,), -math.inf, dtype=torch.float64),
                    lse_tol=torch.zeros(Hq, dtype=torch.float64),
                    p=torch.zeros(Hkv, 0, dtype=torch.float64),
                    p_tol=torch.zeros(Hkv, 0, dtype=torch.float64))
    (kv, _, kbig), (vv, vmid, _) = stored(k), stored(v)
    qd = q.double().view(Hkv, Hq // Hkv, D)
    s = torch.einsum("hgd,nhd->hgn", qd, kv) * scale
    e = abs(scale) * (D + 16) * 2.0 ** -23 * torch.einsum("hgd,nhd->hgn", qd.abs(), kbig).amax(-1)
    lse = torch.logsumexp(s, -1)
    p = (s - lse[..., None]).exp()
    o = torch.einsum("hgn,nhd->hgd", p, vv)
    off = torch.einsum("hgn,nhd->hgd", p, (vv - vmid).abs())
    mid = torch.einsum("hgn,nhd->hgd", p, vmid.abs())
    e3 = e[..., None]
    r = dict(o=o, o_tol=U * o.abs() + (U + 2 * e3 + n * 2.0 ** -23) * off
             + (2 * e3 + n * 2.0 ** -23) * mid,
             lse=lse, lse_tol=e + 2.0 ** -20 * (1 + lse.abs()))
    r = {x: y.reshape(Hq, *y.shape[2:]) for x, y in r.items()}
    r["p"] = p.sum(1)
    r["p_tol"] = ((2.1 * e3 + 2.0 ** -19) * p).sum(1)
    return r


def evict(w, n, budget, recent):
    """Kept slots, ascending, of one (sequence, kv head): fp32 w [slots], n tokens."""
    if n <= budget:
        return list(range(n))
    w = w.tolist()
    early = sorted(range(n - recent), key=lambda i: (-w[i], i))[:budget - recent]
    return sorted(early) + list(range(n - recent, n))
