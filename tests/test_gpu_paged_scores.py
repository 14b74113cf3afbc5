"""mtp_paged_attention over 8 bits where scores are large against their differences, and where a few keys hold
almost all of the softmax, against the fp64 oracle.

Tolerances (derived; A = sum p |v| / sum p).  A part's reference is the largest score that its first block shows, exact but for the
score's own fp32 roundings: the bounds do not grow with the scores beyond those.  Every product here is exact, their fp32 sum S is off by
2^-23 |S| per 16 of hd, and by 4 more such steps for the maximum, the difference and the exponential: a weight by
e = 2^-23 (hd / 16 + 4) S of itself, an output by 2 e A.  A weight is fp16 (2^-11) in three codes: 2^-11 A, and those below 2^-6 of the largest
p_j 2^E_j are off by 2^-26 of it at the most.  The output's rounding is 2^-8 |o|.  lse is off by its score and by some roundings of
its own and of the distance of the scales' exponents: 2^-22 (hd / 8 S + 32 + 4 |lse|)."""
import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib
from oracle import paged
from test_gpu_paged_attention import make_cache, values

pytestmark = pytest.mark.gpu
PAGE = 16


def codes(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def compare(c, table, q, ctx, got, scale, S):
    kv, vv = values(c, "k"), values(c, "v")
    e = np.repeat(c["v_scale"].numpy().astype(int) - 127, 16, -1)[..., None]
    small = [paged.rows(e, table.numpy(), r, n)[..., 0].astype(float) for r, n in enumerate(ctx)]
    o, lse, mass, tiny = paged.attention(q.double().numpy(), kv, vv, table.numpy(), ctx, None, True, scale, small)
    hd = q.shape[-1]
    err = 2.0 ** -23 * (hd / 16 + 4) * S
    go, gl = got["o"].cpu().double().numpy(), got["lse"].cpu().double().numpy()
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * err) * mass + 2.0 ** -26 * tiny + 1e-30
    assert np.isfinite(go).all() and np.isfinite(gl).all()
    worst = (np.abs(go - o) / bound).max()
    assert worst <= 1.01, worst
    assert (np.abs(gl - lse) <= 2.0 ** -22 * (hd / 8 * S + 32 + 4 * np.abs(lse))).all()


def call(c, table, q, ctx, scale):
    assert table.shape[1] * PAGE > 1024  # (not the kernel of short tables)
    got = lib.paged_attention(q.cuda(), **{k: v.cuda() for k, v in c.items()}, page_table=table.cuda(), scale=scale,
                              ctx_len=torch.tensor(ctx, dtype=torch.int32).cuda())
    lib.check_errors()
    return got


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("L,G", [(1, 1), (2, 8), (3, 8), (5, 8)])
@pytest.mark.parametrize("base", [48.0, 32.0, -32.0, -48.0])
def test_large_scores(hd, L, G, base):
    """Scores of +-1024 and +-1536 that differ by some units: a first element of 32 in every query and of `base` in every key."""
    g = torch.Generator().manual_seed(hd + L + G)
    R, per, ctx = 2, 90, [1440, 1101]
    c = make_cache(R * per, 1, hd, PAGE, True, g, 0)
    k = torch.randn((R * per, 1, PAGE, hd), generator=g)
    k[..., 0] = base
    c["k_pages"], c["k_scale"] = codes(k), torch.full_like(c["k_scale"], 127)
    q = (torch.randint(0, 2, (R, L, G, hd), generator=g) - 0.5).to(torch.bfloat16) / 2
    q[..., 0] = 32
    table = torch.randperm(R * per, generator=g).to(torch.int32).view(R, per)
    compare(c, table, q, ctx, call(c, table, q, ctx, 1.0), 1.0, 32 * abs(base) + 64)


@pytest.mark.parametrize("L,G", [(1, 1), (3, 8)])
def test_a_few_keys_hold_almost_all(L, G):
    """Three keys, of values of zero, whose scores are 16.4 above those of 11197 others: the outputs are what those share, each of them
    2^-23.7 of the largest.  (160 requests on the same pages, so that a part has a request's keys from first to last.)"""
    R, hd, per, ctx = 160, 64, 700, 11200
    table = torch.randperm(per, generator=torch.Generator().manual_seed(L)).to(torch.int32).view(1, per)
    c = {n + "_pages": torch.zeros((per, 1, PAGE, hd), dtype=torch.uint8) for n in ("k", "v")}
    c.update({n + "_scale": torch.full((per, 1, 1), 127, dtype=torch.uint8) for n in ("k", "v")})
    c["v_pages"][:] = codes(torch.tensor(1.0))
    for block in range(3):  # of 128 keys
        page = int(table[0, 8 * block])
        c["k_pages"][page, 0, 5, :2] = codes(torch.tensor([16.0, 0.40625]))
        c["v_pages"][page, 0, 5] = 0
    q = torch.zeros((R, L, G, hd), dtype=torch.bfloat16)
    q[..., :2] = 1
    got = call(c, table.expand(R, per).contiguous(), q, [ctx] * R, 1.0)
    compare(c, table, q[:1], [ctx], {k: v[:1] for k, v in got.items()}, 1.0, 17.0)
