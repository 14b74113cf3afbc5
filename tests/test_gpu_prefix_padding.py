"""mtp_prefix_attention where rows of new tokens hold NaN or infinities, as those of a padded
draft do: a token's output is made of the rows that it sees, so the tokens before it are
what they are without it, and only those that see it are not finite.

Tolerances as in test_gpu_prefix_weights.py."""
import numpy as np
import pytest
import torch

from oracle import prefix as op

from test_gpu_prefix import _inputs, _np, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("R,L,H,Hkv,P,T,ctx", [
    (3, 2, 2, 2, 40, 64, [2, 17, 64]),             # few rows, one tile of 16
    (4, 5, 8, 2, 300, 200, [5, 65, 130, 200]),     # two
    (2, 5, 4, 4, 0, 90, [5, 90]),                  # no prefix
    (2, 40, 2, 1, 100, 300, [40, 290]),            # a row tile of 80
    (2, 70, 4, 1, 200, 400, [70, 333]),            # pairs of row tiles
    (80, 5, 8, 2, 130, 60, None),                  # more rows than are joined by four warps each
])
def test_padded_tokens_stay_by_themselves(hd, R, L, H, Hkv, P, T, ctx):
    a = _inputs(R, L, H, Hkv, hd, P, T, R + 5 * L + P, std=0.5)
    if ctx is None:
        ctx = [min(T, L + r % (T - L + 1)) for r in range(R)]
    f = {k: _np(v) for k, v in a.items()}
    rows = sorted({0, 1, R // 2, R - 1})
    o, lse, mass = op.attention(f["q"][rows], f["prefix_k"], f["prefix_v"], f["kv_k"][rows], f["kv_v"][rows],
                                [ctx[r] for r in rows])
    kmax = max(np.abs(f[k]).max() for k in ("prefix_k", "kv_k") if f[k].size)
    S = hd ** -0.5 * np.abs(f["q"][rows]).sum(-1, keepdims=True) * kmax
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -15 + 2.0 ** -20 * (S + 4)) * mass + 1e-30
    real = L - 1 - L // 3  # tokens of the requests that are padded: every second one
    for bad_k, bad_v in ((False, float("inf")), (True, float("nan"))):
        for r in range(0, R, 2):
            at = ctx[r] - L + real
            a["kv_v"][r, at:ctx[r]] = bad_v
            if bad_k:
                a["kv_k"][r, at:ctx[r]] = float("nan")
                a["q"][r, real:] = float("nan")
        got = _run(a, ctx)
        go, gl = _np(got["o"][rows]), _np(got["lse"][rows])
        for i, r in enumerate(rows):
            n = real if r % 2 == 0 else L
            assert (np.abs(go[i, :n] - o[i, :n]) <= bound[i, :n]).all(), (r, bad_v)
            np.testing.assert_allclose(gl[i, :n], lse[i, :n], rtol=1e-5, atol=1e-4)
            assert not np.isfinite(go[i, n:]).any()
