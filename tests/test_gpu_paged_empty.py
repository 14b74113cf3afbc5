"""A step in which no request takes part, and one without rows: nothing is written."""
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,L", [(0, 4), (2, 0), (0, 0)])
@pytest.mark.parametrize("queries", [True, False])
def test_append_and_gather(R, L, queries):
    pages = {n: torch.full((3, 2, 16, 64), 7.0, dtype=torch.bfloat16, device="cuda") for n in ("k_pages", "v_pages")}
    k = torch.ones((R, L, 2, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.zeros((R, 1), dtype=torch.int32, device="cuda")
    ctx = torch.full((R,), 3, dtype=torch.int32, device="cuda")
    f, m = lib.rope_frequencies(64)
    q = lib.kv_append(k, k.clone(), **pages, page_table=table, ctx_len=ctx, inv_freq=f, mscale=m, q=k.repeat(1, 1, 2, 1) if queries else None)
    assert (q.shape == (R, L, 4, 64)) if queries else q is None
    got = lib.kv_gather(**pages, page_table=table, ctx_len=ctx, T=5)
    assert got["k"].shape == (R, 5, 2, 64) and (got["k"][:, :3] == 7).all() and (got["v"][:, 3:] == 0).all()
    assert all((p == 7).all() for p in pages.values())
    lib.check_errors()
