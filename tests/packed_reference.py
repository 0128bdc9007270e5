"""Plain 64-bit attention over packed sequences, its gradients, and bounds on how
far a bf16 kernel's results may be from them.

The bounds count the roundings of the kernels' arithmetic (u = 2^-8, half a bf16
step relative to the value; fp32 accumulation of n products errs by at most
n 2^-24 times the sum of their magnitudes):
  score  e_s = (D + 8) 2^-23 scale sum_d |q_d k_d|       (also bounds the LSE's, plus 2^-20)
  O      u |O| + (u + 2 e_s + n 2^-23) sum_j P |v_j|      P rounded to bf16 for the product
  dV     the same with sum_i P |dO_i|
  dS     u |dS| + P (e_Delta + e_dP) + 2 e_s |dS|
         e_dP = (D + 2) 2^-23 sum |dO v|,  e_Delta = sum_d |dO_d| e_O,d + (D + 2) 2^-23 sum |dO O|
  dQ     u |dQ| + scale sum_j (e_dS + n 2^-23 |dS|) |k_j|;  dK likewise over i
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -8


def mask_of(n, causal=True, window=None):
    wl, wr = (-1, 0 if causal else -1) if window is None else window
    i, j = torch.arange(n)[:, None], torch.arange(n)[None, :]
    m = torch.ones(n, n, dtype=torch.bool)
    if wl >= 0:
        m &= j >= i - wl
    if wr >= 0:
        m &= j <= i + wr
    return m


def one_head(q, k, v, scale, mask, do=None):
    """fp64 [n, D] tensors of one sequence and head pair -> dict of results and bounds."""
    n, D = q.shape
    s = (q @ k.T) * scale
    s = s.masked_fill(~mask, -math.inf)
    lse = torch.logsumexp(s, 1)
    p = (s - lse[:, None]).exp()
    o = p @ v
    e_s = (D + 8) * 2.0 ** -23 * scale * (q.abs() @ k.abs().T).masked_fill(~mask, 0).amax(1)
    a = p @ v.abs()
    r = {"o": o, "lse": lse, "p": p}
    r["o_tol"] = U * o.abs() + (U + 2 * e_s[:, None] + n * 2.0 ** -23) * a
    r["lse_tol"] = e_s + 2.0 ** -20 * (1 + lse.abs())
    if do is None:
        return r
    dp = do @ v.T
    delta = (do * o).sum(1, keepdim=True)
    ds = p * (dp - delta)
    r["dv"] = p.T @ do
    r["dq"] = ds @ k * scale
    r["dk"] = ds.T @ q * scale
    pe = p * (U + 2 * e_s[:, None] + n * 2.0 ** -23)
    r["dv_tol"] = pe.T @ do.abs()  # plus U |dv| once the group's sum is known
    e_dp = (D + 2) * 2.0 ** -23 * (do.abs() @ v.abs().T)
    e_delta = ((do.abs() * r["o_tol"]).sum(1, keepdim=True)
               + (D + 2) * 2.0 ** -23 * (do * o).abs().sum(1, keepdim=True))
    e_ds = (U + 2 * e_s[:, None] + n * 2.0 ** -23) * ds.abs() + p * (e_delta + e_dp)
    r["dq_tol"] = U * r["dq"].abs() + scale * (e_ds @ k.abs())
    r["dk_tol"] = scale * (e_ds.T @ q.abs())
    return r


def packed(q, k, v, bounds, causal=True, window=None, scale=None, do=None):
    """bf16 CPU q [T,Hq,D], k/v [T,Hkv,D] and the sequences' [lo, hi) rows -> fp64
    o, lse [Hq,T] (and dq, dk, dv) with their bounds; rows of no sequence are NaN."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    nan = float("nan")
    out = {"o": torch.full((T, Hq, D), nan, dtype=torch.float64),
           "lse": torch.full((Hq, T), nan, dtype=torch.float64)}
    out |= {n + "_tol": torch.full_like(x, nan) for n, x in list(out.items())}
    if do is not None:
        do = do.double()
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            out[n], out[n + "_tol"] = torch.full_like(x, nan), torch.full_like(x, nan)
    for lo, hi in bounds:
        if hi == lo:
            continue
        mask = mask_of(hi - lo, causal, window)
        for name in ("dk", "dv", "dk_tol", "dv_tol"):
            if name in out:
                out[name][lo:hi] = 0
        for h in range(Hq):
            g = h // (Hq // Hkv)
            r = one_head(q[lo:hi, h], k[lo:hi, g], v[lo:hi, g], scale, mask,
                         None if do is None else do[lo:hi, h])
            for name in ("o", "o_tol", "dq", "dq_tol"):
                if name in out:
                    out[name][lo:hi, h] = r[name]
            for name in ("lse", "lse_tol"):
                out[name][h, lo:hi] = r[name]
            for name in ("dk", "dv", "dk_tol", "dv_tol"):
                if name in out:
                    out[name][lo:hi, g] += r[name]
        for name in ("dk", "dv"):
            if name in out:
                out[name + "_tol"][lo:hi] += U * out[name][lo:hi].abs()
    return out


def assert_within(got, ref, tol, what):
    got = got.detach().cpu().double()
    live = ~torch.isnan(ref)
    assert bool(torch.isfinite(got[live]).all()), f"{what}: not finite"
    over = (got[live] - ref[live]).abs() - (tol[live] + 1e-30)
    assert not over.numel() or over.max() <= 0, (
        f"{what}: off by {(got[live] - ref[live]).abs().max():.3e}, "
        f"worst {over.max():.3e} over its bound")
