"""The shared-prefix attention oracle against the draft oracle's attention over
one concatenated cache, and by hand."""
import numpy as np

from oracle import draft as od
from oracle import prefix as op


def test_equals_attention_over_one_cache():
    rng = np.random.default_rng(0)
    R, H, hd, P, T = 3, 4, 8, 10, 6
    q = rng.standard_normal((R, 1, H, hd))
    pk, pv = rng.standard_normal((2, P, H, hd))
    kk, kv = rng.standard_normal((2, R, T, H, hd))
    ctx = [0, 4, 6]
    o, lse, mass = op.attention(q, pk, pv, kk, kv, ctx)
    for r in range(R):
        k = np.concatenate([pk, kk[r, :ctx[r]]]).reshape(-1, H * hd)
        v = np.concatenate([pv, kv[r, :ctx[r]]]).reshape(-1, H * hd)
        np.testing.assert_allclose(o[r, 0].reshape(-1), od.cached_attention(q[r, 0].reshape(-1), k, v, H, hd), rtol=1e-12)
    assert (mass >= np.abs(o) - 1e-12).all() and np.isfinite(lse).all()


def test_causal_rows_grouped_heads_and_empty_rows():
    """Two query heads on one key head; with uniform scores a token's output is
    the mean of the values that it sees: itself and what precedes it."""
    q = np.zeros((1, 3, 2, 4))
    kk = np.zeros((1, 5, 1, 4))
    kv = np.arange(5.0)[None, :, None, None] * np.ones((1, 5, 1, 4))
    none = np.zeros((0, 1, 4))
    o, lse, _ = op.attention(q, none, none, kk, kv, [4])
    np.testing.assert_allclose(o[0, :, 1, 0], [0.5, 1.0, 1.5])  # rows 0..1, 0..2, 0..3
    np.testing.assert_allclose(lse[0, :, 0], np.log([2, 3, 4]))
    o, lse, _ = op.attention(q, none, none, kk, kv, [4], causal=False)
    np.testing.assert_allclose(o[0, :, 0, 0], 1.5)
    o, lse, _ = op.attention(q, none, none, kk, kv, [1])
    assert (o == 0).all() and lse[0, :2].tolist() == [[-np.inf] * 2] * 2 and lse[0, 2, 0] == 0
