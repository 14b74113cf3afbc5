"""Outputs of mtp_rope and mtp_kv_append that lie beside their inputs, or between other rows, are taken, with the results of outputs apart
(what is refused: test_abi_paged_overlap.py)."""
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,H,on,oh", [
    (3, 2, 256, 128), (2, 4, 512, 128), (8, 3, 128, 1024), (3, 3, 384, 1152), (4, 3, 896, 384), (7, 5, 1000, 136), (100, 7, 136, 13600),
    (4, 300, 128, 512), (3, 2, 384, 256), (2, 3, 640, 256)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_rows_between_one_another(N, H, on, oh, in_place):
    """Strides in either order, and rows of one position between those of others."""
    at = (torch.arange(N)[:, None] * on + torch.arange(H) * oh).flatten().sort().values
    assert (at.diff() >= 128).all()  # rows apart
    g = torch.Generator().manual_seed(N + H)
    x = torch.randn((N, H, 128), generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 4000, (N,), generator=g, dtype=torch.int32).cuda()
    f, m = lib.rope_frequencies(64)
    want = lib.rope(x, pos, f, m)
    memory = torch.full(((N - 1) * on + (H - 1) * oh + 128,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = memory.as_strided((N, H, 128), (on, oh, 1))
    if in_place:
        out.copy_(x)
        lib.rope(out, pos, f, m, out=out)
    else:
        lib.rope(x, pos, f, m, out=out)
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert (memory == 7.0).all()
    lib.check_errors()


@pytest.mark.parametrize("H", [2, 8])
def test_append_with_queries_beside_inputs(H):
    """One buffer for k, v, q and q_out, one behind the other, in any order, and q in place."""
    R, L, Hkv, hd = 2, 3, 2, 64
    g = torch.Generator().manual_seed(H)
    data = {n: torch.randn((R, L, h, hd), generator=g).to(torch.bfloat16).cuda() for n, h in (("k", Hkv), ("v", Hkv), ("q", H))}
    f, m = lib.rope_frequencies(hd)
    table = torch.arange(R, dtype=torch.int32).view(R, 1).cuda()
    ctx = torch.tensor([5, 16], dtype=torch.int32).cuda()
    want = None
    for order in (("k", "v", "q", "q_out"), ("q_out", "q", "k", "v"), ("k", "q_out", "v", "q"), ("v", "k", "q")):
        sizes = [(H if n[0] == "q" else Hkv) * R * L * hd for n in order]
        parts = dict(zip(order, torch.zeros(sum(sizes), dtype=torch.bfloat16, device="cuda").split(sizes)))
        t = {n: parts[n].view(R, L, -1, hd) for n in order}
        for n in data:
            t[n].copy_(data[n])
        pages = {n: torch.zeros((R, Hkv, 16, hd), dtype=torch.bfloat16, device="cuda") for n in ("k_pages", "v_pages")}
        got = lib.kv_append(t["k"], t["v"], **pages, page_table=table, ctx_len=ctx, inv_freq=f, mscale=m, q=t["q"],
                            q_out=t.get("q_out", t["q"]))
        lib.check_errors()
        now = (got.clone(), pages["k_pages"], pages["v_pages"])
        assert want is None or all(torch.equal(a, b) for a, b in zip(now, want))
        want = now
        assert all(torch.equal(t[n], data[n]) for n in ("k", "v"))
