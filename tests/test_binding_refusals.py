"""What the binding refuses without a GPU: a weight block whose tensors the kernels cannot
read must not get as far as its addresses."""
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib, synth


@pytest.fixture(scope="module")
def block():
    return synth.make_int4_block(synth.make_draft_inputs(synth.DRAFT_SMALL, 1)["weights"], 64)


def test_4bit_weights_on_the_cpu_are_refused(block):
    with pytest.raises(lib.MtpError, match="CUDA"):
        lib.Int4Block(block, 64, synth.DRAFT_SMALL)


def test_gemm_int4w_refuses_weights_on_the_cpu(block):
    q, s, z = block["wq"]
    with pytest.raises(lib.MtpError):
        lib.gemm_int4w(torch.zeros(1, 256, dtype=torch.bfloat16), q, s, z, group=64)
