"""Draft steps at the batch sizes that they are for, where other kernels run than for four or
five requests: 4-bit maps on three and four tiles of 8 tokens, grouped launches among them; a
prefix of 17 to 32 rows per key head on row tiles, its records joined one row per warp and left
unnormalised between those of the own caches.  bf16, FP8 and 4-bit maps.

Bars: those of the FP8 draft steps (test_gpu_fp8.py: h, total variation, and 5e-3 max(q)
per entry of q, two rounding flips of the normalised head input at their largest).  The maps'
and the attention's own errors are far smaller: the 4-bit products are exact to fp32 sums, the
prefix's weights to 2^-15, where one bf16 step of the attention's output is 2^-8."""
import dataclasses

import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib, synth
from oracle import chain as oc
from oracle import fp8 as of
from oracle import int4 as oi

from test_gpu_draft import _np, check
from test_gpu_draft_ext import _dev, _draws, _inputs, _oracle
from test_gpu_fp8 import Q_BAR

pytestmark = pytest.mark.gpu
# 40 heads: 1280 rows at R = 32, more than eight per SM
MANY_HEADS = synth.DraftConfig(name="draft_many_heads", R=32, ctx=70, d=2560, n_heads=40, head_dim=64, ffn=320, V=500,
                               w_std=0.02, gain_std=0.1)


def _forms(inp, form):
    W = oc.weights_to_numpy(inp["weights"])
    if form == "int4":
        i4 = synth.make_int4_block(inp["weights"], 64, False)
        W = oi.draft_weights(W, {k: (v[0].numpy(), _np(v[1]), v[2].numpy()) for k, v in i4.items()}, 64)
        return W, dict(int4={k: tuple(t.cuda() for t in v) for k, v in i4.items()}, int4_group=64)
    if form == "fp8":
        f8 = synth.make_fp8_block(inp["weights"])
        W = of.draft_weights(W, {k: (_np(q), _np(s)) for k, (q, s) in f8.items()})
        return W, dict(fp8={k: (q.cuda(), s.cuda()) for k, (q, s) in f8.items()})
    return W, {}


def _run(cfg, prefix, form, seed):
    ctx = [(r * 37) % (cfg.ctx + 1) for r in range(cfg.R)]  # empty ones among them
    inp, pk, pv = _inputs(cfg, seed, ctx, prefix)
    W, kw = _forms(inp, form)
    dev, w = _dev(inp)
    step = lib.DraftStep(cfg, w, prefix_len=prefix, **kw)
    h = torch.empty((cfg.R, cfg.d), dtype=torch.bfloat16, device="cuda")
    rows = dict(prefix_k=pk.cuda(), prefix_v=pv.cuda()) if prefix else {}
    g = step(**dev, seed=seed, offset=2, h_out=h, **rows)
    lib.check_errors()
    g = {k: _np(v) for k, v in g.items()}
    r = _oracle(cfg, inp, pk, pv, W, seed, 2)
    check(g, r, list(range(cfg.R)), qbar=Q_BAR)
    _draws(cfg, g, r, seed, 2)
    return inp, pk, pv, g


@pytest.mark.parametrize("form", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("base,R,prefix", [(synth.DRAFT_SMALL, 17, 333), (synth.DRAFT_SMALL, 25, 130), (synth.DRAFT_SMALL, 32, 1),
                                           (synth.DRAFT_SMALL_HD128, 32, 700), (synth.DRAFT_SMALL_HD128, 9, 64), (synth.DRAFT_SMALL, 5, 127),
                                           (synth.DRAFT_SMALL_HD128, 4, 700)])
def test_batches_on_a_shared_prefix(base, R, prefix, form):
    _run(dataclasses.replace(base, R=R), prefix, form, 40 + R)


@pytest.mark.parametrize("R", [9, 16, 18, 31])
def test_batches_with_4bit_maps(R):
    _run(dataclasses.replace(synth.DRAFT_SMALL, R=R), 0, "int4", 50 + R)


@pytest.mark.parametrize("form", ["bf16", "int4"])
def test_many_rows_to_join(form):
    _run(MANY_HEADS, 150, form, 60)


@pytest.mark.parametrize("base,R,prefix", [(synth.DRAFT_SMALL, 32, 260), (synth.DRAFT_SMALL_HD128, 12, 400)])
def test_prefix_rows_in_the_own_caches(base, R, prefix):
    """The same step with the prefix's rows at the head of every request's own cache."""
    cfg = dataclasses.replace(base, R=R)
    inp, pk, pv, g = _run(cfg, prefix, "int4", 70)
    _, kw = _forms(inp, "int4")
    whole = dataclasses.replace(cfg, ctx=cfg.ctx + prefix)
    dev, w = _dev(inp)
    for k, p in (("kv_k", pk), ("kv_v", pv)):
        dev[k] = torch.cat([p.cuda().expand(R, *p.shape), dev[k]], 1).contiguous()
    dev["ctx_len"] = dev["ctx_len"] + prefix
    alone = {k: _np(v) for k, v in lib.DraftStep(whole, w, **kw)(**dev, seed=70, offset=2).items()}
    assert (np.abs(g["q"] - alone["q"]).max(1) <= Q_BAR * alone["q"].max(1)).all()
