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


def test_maps_in_another_form_need_no_bf16_ones():
    """include/mtp.h: with FP8 or 4-bit maps the weights' own are not read and may be null."""
    w = synth.make_draft_inputs(synth.DRAFT_SMALL, 1)["weights"]
    rest = {k: v for k, v in w.items() if k not in lib.FP8_LINEAR_MAPS}
    views = lib.ChainWeights(rest, 1, lib.FP8_LINEAR_MAPS).struct
    assert views.hnorm[0] == w["hnorm"][0].data_ptr() and not views.wq and not views.w_down
    with pytest.raises(KeyError):
        lib.ChainWeights(rest, 1)
