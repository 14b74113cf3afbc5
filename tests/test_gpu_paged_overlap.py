"""Outputs of mtp_rope whose rows lie between one another are taken, with the results of outputs apart
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
