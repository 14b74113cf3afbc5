"""Draft steps whose linear maps are in FP8 or in 4 bits: the bf16 maps need not exist."""
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib, synth

pytestmark = pytest.mark.gpu
CFG = synth.DRAFT_SMALL


def _state():
    inp = synth.make_draft_inputs(CFG, 2)
    dev = {k: v.cuda() for k, v in inp.items() if k != "weights"}
    w = {k: ([t.cuda() for t in v] if isinstance(v, list) else v.cuda()) for k, v in inp["weights"].items()}
    i4 = {k: tuple(None if t is None else t.cuda() for t in v) for k, v in synth.make_int4_block(inp["weights"], 64).items()}
    f8 = {k: tuple(t.cuda() for t in v) for k, v in synth.make_fp8_block(inp["weights"]).items()}
    return dict(dev, seed=3, offset=0), w, i4, f8


def test_bf16_maps_may_be_left_out():
    kw, w, i4, f8 = _state()
    rest = {k: v for k, v in w.items() if k not in lib.FP8_LINEAR_MAPS}
    want, got = lib.DraftStep(CFG, w, int4=i4, int4_group=64)(**kw), lib.DraftStep(CFG, rest, int4=i4, int4_group=64)(**kw)
    assert torch.equal(got["q"], want["q"]) and torch.equal(got["y"], want["y"])
    got = lib.DraftRound(CFG, rest, 2, int4=i4, int4_group=64)(**kw)
    assert torch.equal(got["q"][:, 0], want["q"])
    # the FP8 maps' partial sums are added in any order: the same to the draft bars
    want, got = lib.DraftStep(CFG, w, fp8=f8)(**kw), lib.DraftStep(CFG, rest, fp8=f8)(**kw)
    assert ((got["q"] - want["q"]).abs().sum(1) < 1e-2).all()
    lib.check_errors()
    with pytest.raises((lib.MtpError, KeyError)):
        lib.DraftStep(CFG, rest)


def test_weights_are_checked():
    kw, w, i4, _ = _state()
    for name, bad in (("head", w["head"].cpu()), ("head", w["head"][:-1]), ("embed", w["embed"].float()), ("out_norm", w["out_norm"][:-1]),
                      ("hnorm", [w["hnorm"][0][:-1]]), ("wq", [w["wq"][0].cpu()]), ("w_gate", [w["w_down"][0]]),
                      ("w_up", [w["w_down"][0].t()]), ("hnorm", [])):
        with pytest.raises(lib.MtpError):
            lib.DraftStep(CFG, {**w, name: bad})
    with pytest.raises(lib.MtpError):
        lib.DraftStep(CFG, w, device="cpu")
    lib.DraftStep(CFG, {**w, "another": torch.zeros(3)})  # not the step's
    lib.DraftStep(CFG, {**w, "wq": [w["wq"][0].cpu()]}, int4=i4, int4_group=64)  # not read
