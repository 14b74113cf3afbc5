"""What the binding refuses of tensors on a GPU."""
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib, synth

pytestmark = pytest.mark.gpu


def _block():
    return synth.make_int4_block(synth.make_draft_inputs(synth.DRAFT_SMALL, 1)["weights"], 64, False)


@pytest.mark.parametrize("where", [0, 1, 2])
def test_a_4bit_block_is_on_one_gpu_as_a_whole(where):
    block = {k: tuple(t.cuda() for t in v) for k, v in _block().items()}
    lib.Int4Block(block, 64, synth.DRAFT_SMALL)
    block["wo"] = tuple(t.cpu() if i == where else t for i, t in enumerate(block["wo"]))
    with pytest.raises(lib.MtpError):
        lib.Int4Block(block, 64, synth.DRAFT_SMALL)


def test_prefix_attention_workspaces():
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    args = (n(2, 1, 4, 64), n(300, 2, 64), n(300, 2, 64))
    want = lib.prefix_attention(*args)
    size = 1 << 22
    for ws in (torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty(size // 4, device="cuda")):
        assert torch.equal(lib.prefix_attention(*args, ws=ws)["o"], want["o"])
    for ws in (torch.empty(size, dtype=torch.uint8), torch.empty(2 * size, dtype=torch.uint8, device="cuda")[::2],
               torch.empty(16, dtype=torch.uint8, device="cuda"), torch.empty(size + 1, dtype=torch.uint8, device="cuda")[1:]):
        with pytest.raises(lib.MtpError):
            lib.prefix_attention(*args, ws=ws)
