"""Plain 64-bit attention under a window with sinks over packed sequences, with the bounds
of packed_reference."""
from __future__ import annotations

import math

import torch

from packed_reference import U, mask_of, one_head


def sink_mask(n, window, sinks):
    """[n, n]: the window, and the first `sinks` keys behind its left side."""
    m = mask_of(n, False, window)
    j = torch.arange(n)[None, :]
    i = torch.arange(n)[:, None]
    wl, _ = window
    return m | ((j < sinks) & (j < i - wl)) if wl >= 0 else m


def packed_sinks(q, k, v, bounds, window, sinks, scale=None, do=None):
    """As packed_reference.packed: bf16 CPU tensors -> fp64 results with their bounds.  (The
    bounds take a positive scale; a negative one is the positive one with -k.)"""
    if scale is not None and scale < 0:
        r = packed_sinks(q, -k, v, bounds, window, sinks, -scale, do)
        if do is not None:
            r["dk"] = -r["dk"]
        return r
    T, Hq, D = q.shape
    group = Hq // k.shape[1]
    scale = 1 / math.sqrt(D) if scale is None else scale
    q, k, v = q.double(), k.double(), v.double()
    nan = float("nan")
    like = {"o": q, "lse": torch.empty(Hq, T)}
    if do is not None:
        do = do.double()
        like |= {"dq": q, "dk": k, "dv": v}
    out = {n: torch.full(x.shape, nan, dtype=torch.float64) for n, x in like.items()}
    out |= {n + "_tol": torch.full_like(x, nan) for n, x in list(out.items())}
    for lo, hi in bounds:
        if hi == lo:
            continue
        mask = sink_mask(hi - lo, window, sinks)
        for name in ("dk", "dv", "dk_tol", "dv_tol"):
            if name in out:
                out[name][lo:hi] = 0
        for h in range(Hq):
            r = one_head(q[lo:hi, h], k[lo:hi, h // group], v[lo:hi, h // group], scale, mask,
                         None if do is None else do[lo:hi, h])
            for name in ("o", "o_tol", "dq", "dq_tol"):
                if name in out:
                    out[name][lo:hi, h] = r[name]
            out["lse"][h, lo:hi], out["lse_tol"][h, lo:hi] = r["lse"], r["lse_tol"]
            for name in ("dk", "dv", "dk_tol", "dv_tol"):
                if name in out:
                    out[name][lo:hi, h // group] += r[name]
        for name in ("dk", "dv"):
            if name in out:
                out[name + "_tol"][lo:hi] += U * out[name][lo:hi].abs()
    return out
