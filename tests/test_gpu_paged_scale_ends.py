"""Scales at the ends of their range in a cache of 8 bits: 2^127 (254) in a block that goes on, and bytes outside 1..254, which
are taken as the nearest one by everything that reads them."""
import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib

pytestmark = pytest.mark.gpu


def cache(scale, code=0x38):  # 0x38: 1.0
    c = {n + "_pages": torch.full((1, 1, 16, 64), code, dtype=torch.uint8, device="cuda") for n in ("k", "v")}
    c.update({n + "_scale": torch.full((1, 1, 1), scale, dtype=torch.uint8, device="cuda") for n in ("k", "v")})
    c["page_table"] = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    return c


@pytest.mark.parametrize("scale,kept", [(254, 254), (253, 253), (255, 254)])
def test_a_block_of_the_largest_scale_goes_on(scale, kept):
    """What was there keeps its scale; a row of 2^124 is the code of 2^-3 of it, one of 3 is zero."""
    c = cache(scale)
    k = torch.full((1, 2, 1, 64), 2.0 ** 124, dtype=torch.bfloat16, device="cuda")
    k[0, 1] = 3.0
    lib.kv_append(k, k.clone(), **c, ctx_len=torch.tensor([7], dtype=torch.int32, device="cuda"))
    lib.check_errors()
    for n in ("k", "v"):
        assert int(c[n + "_scale"]) == kept
        value = c[n + "_pages"].view(torch.float8_e4m3fn).float().cpu()[0, 0, :, 0].double() * 2.0 ** (kept - 127)
        np.testing.assert_array_equal(value[:7], [2.0 ** (kept - 127)] * 5 + [2.0 ** 124, 0.0])


@pytest.mark.parametrize("scale,taken", [(0, 1), (255, 254)])
def test_bytes_out_of_range(scale, taken):
    """Reading back and attention agree on them."""
    ctx = torch.tensor([9], dtype=torch.int32, device="cuda")
    a, b = (lib.kv_gather(**cache(s), ctx_len=ctx, T=16) for s in (scale, taken))
    assert torch.equal(a["k"], b["k"]) and torch.equal(a["v"], b["v"]) and (a["k"][0, :9] != 0).all()
    q = torch.ones((1, 1, 1, 64), dtype=torch.bfloat16, device="cuda") * 2.0 ** -120
    for wide in (1, 70):
        got = []
        for s in (scale, taken):
            c = cache(s)
            c["v_scale"][:] = 127
            c["page_table"] = torch.zeros((1, wide), dtype=torch.int32, device="cuda")
            got.append(lib.paged_attention(q, **c, ctx_len=ctx))
        assert torch.equal(got[0]["o"], got[1]["o"]) and torch.equal(got[0]["lse"], got[1]["lse"])
        assert (got[0]["o"] == 1).all()
    lib.check_errors()
