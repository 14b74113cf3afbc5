"""4-bit group-scaled weights -- oracle, test infrastructure only.

"M7.6 - DeepSeek MTP" §0x03C leaves the runtime's weight representation open;
this one keeps two 4-bit codes per byte (the even column in the low half) and
per row and group of columns one bf16 scale and one zero point (8 where none
is given):

    W[m, k] = (code[m, k] - zero[m, k // group]) * scale[m, k // group]

taken exactly (a 5-bit integer times 8 significant bits)."""
from __future__ import annotations

import numpy as np

LINEAR_MAPS = ("eh_proj", "wq", "wk", "wv", "wo", "w_gate", "w_up", "w_down")


def dequantize(q, scale, zero, group):
    """W [n, K] in fp64 from q uint8 [n, K/2], scale [n, ceil(K/group)], zero likewise or None."""
    q = np.asarray(q)
    n, K = q.shape[0], 2 * q.shape[1]
    codes = np.empty((n, K), dtype=np.float64)
    codes[:, 0::2] = q & 15
    codes[:, 1::2] = q >> 4
    col = np.arange(K) // group
    z = 8.0 if zero is None else (np.asarray(zero) & 15).astype(np.float64)[:, col]
    return (codes - z) * np.asarray(scale, dtype=np.float64)[:, col]


def draft_weights(weights: dict, int4: dict, group: int) -> dict:
    """A draft step's weight dict with its linear maps replaced by the dequantised ones."""
    out = dict(weights)
    for name in LINEAR_MAPS:
        q, s, z = int4[name]
        out[name] = [dequantize(q, s, z, group)]
    return out
