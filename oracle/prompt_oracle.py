"""fp64 oracle of attention over whole prompts (numpy; test infrastructure)."""
from __future__ import annotations

import math

import numpy as np


def prompt_attention(q, k, v, cu_q, cu_k, scale, causal):
    """q [Tq, H, d]; k, v [Tk, Hkv, d]. Returns (out, lse [H, Tq], abs-weighted mean
    of v, largest sum |q||k| * scale over the keys a row sees [Tq, H]). Rows past
    cu_q[-1] are zeros."""
    T, H, d = q.shape
    G = H // k.shape[1]
    out, av = np.zeros((T, H, d)), np.zeros((T, H, d))
    lse, mag = np.full((H, T), -math.inf), np.zeros((T, H))
    for g in range(len(cu_q) - 1):
        a, b, c, e = cu_q[g], cu_q[g + 1], cu_k[g], cu_k[g + 1]
        n, m = b - a, e - c
        if n == 0 or m == 0:
            continue
        seen = np.arange(m)[None, :] <= np.arange(n)[:, None] + (m - n) if causal else np.ones((n, m), bool)
        some = seen.any(1)
        for h in range(H):
            kk, vv = k[c:e, h // G], v[c:e, h // G]
            with np.errstate(invalid="ignore"):
                z = np.where(seen, scale * (q[a:b, h] @ kk.T), -math.inf)
                terms = np.where(seen, scale * (np.abs(q[a:b, h]) @ np.abs(kk).T), 0.0)
            top = np.where(some, z.max(1), 0.0)
            p = np.where(seen, np.exp(z - top[:, None]), 0.0)
            total = np.where(some, p.sum(1), 1.0)
            p /= total[:, None]
            out[a:b, h], av[a:b, h] = p @ vv, p @ np.abs(vv)
            lse[h, a:b] = np.where(some, top + np.log(total), -math.inf)
            mag[a:b, h] = terms.max(1)
    return out, lse, av, mag
