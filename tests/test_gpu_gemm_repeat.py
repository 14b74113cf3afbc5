"""Chain states are the same bits every time, also where a GEMM's last column tile
ends past the matrix (d = 384): pieces of the tile that are not stored must not let a
staging box be written while an earlier store still reads it.  (That lost rows of one
64-column piece in about one call in 200, more where memory was busy.)"""
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["small_bf16_hd128", "small_bf16_D2"])
def test_repeated_calls_are_equal(name):
    cfg = synth.CHAIN_CONFIGS[name]
    inp = synth.make_chain_inputs(cfg, seed=13)
    dev = {k: v.cuda() for k, v in inp.items() if k != "weights"}
    w = {k: ([t.cuda() for t in v] if isinstance(v, list) else v.cuda()) for k, v in inp["weights"].items()}
    chain = lib.Chain(cfg, w)
    big = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    args = [dev[k] for k in ("tokens", "seg", "pos", "h0")]
    h = torch.zeros((cfg.D, cfg.B, cfg.T, cfg.d), dtype=torch.bfloat16, device="cuda")
    first, wrong = None, torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(1500):
        chain.ws.zero_()
        if i % 3 == 0:
            big.zero_()
        if i % 2:
            torch.cuda.synchronize()
        if i % 4:
            chain.loss(*args, row_loss=True, h_out=h)
        else:
            chain.forward(*args, h_out=h)
        if first is None:
            first = h.clone()
        wrong += (h.view(torch.int16) != first.view(torch.int16)).any()
    lib.check_errors()
    assert int(wrong) == 0, f"{int(wrong)} of 1500 calls differ"
