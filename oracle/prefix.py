"""Attention over a shared prefix and each request's own cache -- oracle, test
infrastructure only.

"M7.6 - DeepSeek MTP" §0x09A: the module's attention reads its own K/V cache.
Sharing a prefix changes where keys are kept, not what is computed: the softmax
runs over the concatenation of the prefix rows and the request's own rows.  One
(request, token, head) at a time, in fp64.
"""
from __future__ import annotations

import numpy as np


def attention(q, prefix_k, prefix_v, kv_k, kv_v, ctx_len, causal=True, scale=None):
    """q [R, L, H, hd]; prefix [P, Hkv, hd]; own cache [R, T, Hkv, hd] of
    ctx_len[r] rows, the last L of them the new tokens'.  Returns (o, lse, mass):
    mass = Σ p |v| / Σ p, the scale that rounding p acts on."""
    q = np.asarray(q, dtype=np.float64)
    R, L, H, hd = q.shape
    Hkv = prefix_k.shape[1]
    scale = hd ** -0.5 if scale is None else scale
    o, mass = np.zeros((R, L, H, hd)), np.zeros((R, L, H, hd))
    lse = np.full((R, L, H), -np.inf)
    for r in range(R):
        for i in range(L):
            n = int(ctx_len[r]) - ((L - 1 - i) if causal else 0)
            n = max(0, n)
            for h in range(H):
                g = h // (H // Hkv)
                k = np.concatenate([prefix_k[:, g], kv_k[r, :n, g]]).astype(np.float64)
                v = np.concatenate([prefix_v[:, g], kv_v[r, :n, g]]).astype(np.float64)
                if len(k) == 0:
                    continue
                s = (k @ q[r, i, h]) * scale
                m = s.max()
                p = np.exp(s - m)
                lse[r, i, h] = m + np.log(p.sum())
                o[r, i, h] = (p / p.sum()) @ v
                mass[r, i, h] = (p / p.sum()) @ np.abs(v)
    return o, lse, mass
