"""mtp_prefix_attention: the softmax weights enter the product with the values as two
bf16 parts.

Tolerance (derived).  p_hi, p's upper 16 bits, leaves p - p_hi of less than 2^-7 p,
exact in fp32; p_lo = bf16(p - p_hi) is off by at most 2^-8 of that.  A weight is so
off by 2^-15 of itself, the output by 2^-15 A, A = Σ p |v| / Σ p; its own rounding to
bf16 is 2^-8 |o| at most.  The scores' error (fp32 sums of exact products, hd/16 + 4 steps
of 2^-23 on S = scale Σ |q k|) and the exponential's are covered by 2^-20 (S + 4) A.
A single bf16 part (2^-8 A) is far outside where values cancel, |o| << A."""
import numpy as np
import pytest
import torch

from oracle import prefix as op

from test_gpu_prefix import _inputs, _np, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("R,L,H,Hkv,P,T,ctx", [
    (4, 1, 2, 2, 300, 64, [0, 1, 63, 64]),      # few rows: prefix and own caches
    (3, 16, 2, 2, 50, 700, [16, 31, 700]),
    (2, 8, 8, 2, 0, 400, [8, 400]),
    (17, 1, 2, 2, 333, 40, None),               # 17 rows on the prefix
    (16, 1, 8, 2, 1200, 70, None),              # 64
    (1, 11, 6, 2, 500, 900, [899]),             # 33 rows on the prefix and on the own cache
    (3, 32, 4, 2, 0, 1000, [32, 500, 999]),     # 64 rows over own caches, causal across blocks
    (40, 5, 4, 2, 700, 20, None),               # pairs of row tiles and a single one
    (2, 70, 4, 1, 200, 400, [70, 333]),         # two row tiles over an own cache
    (2, 40, 2, 1, 0, 1000, [40, 999]),          # one
])
def test_weights_are_kept(hd, R, L, H, Hkv, P, T, ctx):
    a = _inputs(R, L, H, Hkv, hd, P, T, 3 * R + L + P, std=0.5)
    if ctx is None:
        ctx = [min(T, L + r % (T - L + 1)) for r in range(R)]
    got = _run(a, ctx)
    f = {k: _np(v) for k, v in a.items()}
    o, _, mass = op.attention(f["q"], f["prefix_k"], f["prefix_v"], f["kv_k"], f["kv_v"], ctx)
    kmax = max(np.abs(f[k]).max() for k in ("prefix_k", "kv_k") if f[k].size)
    S = hd ** -0.5 * np.abs(f["q"]).sum(-1, keepdims=True) * kmax
    bad = np.abs(_np(got["o"]) - o) - (2.0 ** -8 * np.abs(o) + (2.0 ** -15 + 2.0 ** -20 * (S + 4)) * mass + 1e-30)
    assert (bad <= 0).all(), (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
