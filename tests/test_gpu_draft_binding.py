"""DraftStep and DraftRound on streams of the caller's, and what they refuse: inputs and
outputs that the kernels would read or write past their ends."""
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib, synth

pytestmark = pytest.mark.gpu
CFG = synth.DRAFT_SMALL


def _state(gamma):
    inp = synth.make_draft_inputs(CFG, 2)
    dev = {k: v.cuda() for k, v in inp.items() if k != "weights"}
    w = {k: ([t.cuda() for t in v] if isinstance(v, list) else v.cuda()) for k, v in inp["weights"].items()}
    i4 = {k: tuple(None if t is None else t.cuda() for t in v) for k, v in synth.make_int4_block(inp["weights"], 64).items()}
    obj = lib.DraftStep(CFG, w, int4=i4, int4_group=64) if gamma is None else lib.DraftRound(CFG, w, gamma, int4=i4, int4_group=64)
    return obj, dict(dev, seed=3, offset=0)


@pytest.mark.parametrize("gamma", [None, 2])
def test_outputs_belong_to_the_launching_stream(gamma):
    """A block that the current stream has released is not handed to a call on another
    stream, whose kernels would write it while the current one may still use it."""
    call, kw = _state(gamma)
    want = call(**kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    freed = [torch.empty_like(want[k]) for k in ("q", "y")]
    at = {t.data_ptr() for t in freed}
    del freed
    got = call(**kw, stream=side)
    side.synchronize()
    assert not at & {got[k].data_ptr() for k in ("q", "y")}
    assert torch.equal(got["q"], want["q"]) and torch.equal(got["y"], want["y"])
    lib.check_errors()


@pytest.mark.parametrize("gamma", [None, 2])
def test_refusals(gamma):
    call, kw = _state(gamma)
    R, V, d = CFG.R, CFG.V, CFG.d
    rows = (R,) if gamma is None else (R, gamma)
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    good = {"q": f(*rows, V), "y": i(*rows)}
    for bad in (dict(frontier=kw["frontier"][:-1]), dict(frontier=kw["frontier"].cpu()), dict(pos=kw["pos"][:1]),
                dict(pos=kw["pos"].long()), dict(ctx_len=kw["ctx_len"][:-1]), dict(parent_hidden=kw["parent_hidden"][:, : d // 2].contiguous()),
                dict(parent_hidden=kw["parent_hidden"][:-1]), dict(kv_k=kw["kv_k"][:-1]), dict(kv_v=kw["kv_v"].cpu()), dict(pos=None),
                dict(out={**good, "q": f(*rows, V - 1)}), dict(out={**good, "q": f(R - 1, *rows[1:], V)}), dict(out={**good, "y": i(R - 1, *rows[1:])}),
                dict(out={**good, "y": f(*rows)}), dict(out={**good, "q": good["q"].cpu()}), dict(out={**good, "q": f(*rows, 2 * V)[..., ::2]}),
                dict(h_out=b(R - 1, *rows[1:], d)), dict(h_out=f(*rows, d)), dict(parent_hidden=kw["parent_hidden"].cpu())):
        with pytest.raises(lib.MtpError):
            call(**{**kw, **bad})
    call(**kw, out=good, h_out=b(*rows, d))
    lib.check_errors()
