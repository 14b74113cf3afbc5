"""Draft steps and rounds with 4-bit linear maps and with a prefix that all
requests share (mtp_draft_round_ext), against the draft oracle: on the exactly
dequantised weights, and on caches that begin with the prefix's rows.

Bars: h within 2e-2 + 2e-2 |h|; q within total variation 5e-3 and 1.15e-2 max(q)
per entry.  q moves with the bf16 rounding flips of the normalised head input x: a
flip of element j moves logit v by W_jv step_j, and q_v by that share of itself.
Values of unit variance have a mean squared step of 3.3e-5 (2^-7 in [1, 2), 2^-6 in
[2, 4), 2^-8 in [1/2, 1), ..), and sum_j W_jv^2 = 256 * 0.05^2 = 0.64.  A flip's
chance is the two sides' difference before the rounding in steps, which is itself
the sum of flips earlier in the block, of some quarter step: a quarter of the
elements flip, a logit's standard deviation is sqrt(3.3e-5 * 0.64 / 4) = 2.3e-3, and
the bar five of them.  (5e-3, two flips at most, was too narrow: 2.2 of them, over
some 50 rows of 777 entries.  The prefix's softmax weights are bf16, which moves the
attention output by at most half a bf16 step of its own scale before it is rounded to
bf16 anyway: another source of flips, no larger.)"""
import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib, synth
from oracle import chain as oc
from oracle import draft as od
from oracle import int4 as oi
from oracle import verify as ov

from test_gpu_draft import _check_round, _np, check

pytestmark = pytest.mark.gpu
Q_BAR = 1.15e-2


def _inputs(cfg, seed, ctx, prefix):
    """Draft inputs whose first `prefix` cache rows are the same for every request."""
    inp = synth.make_draft_inputs(cfg, seed)
    ctx = torch.tensor(ctx, dtype=torch.int32)
    g = torch.Generator().manual_seed(seed + 50)
    pk, pv = (torch.randn((prefix, cfg.d), generator=g).to(torch.bfloat16) for _ in range(2))
    inp["ctx_len"], inp["pos"] = ctx, ctx + prefix
    return inp, pk, pv


def _dev(inp):
    dev = {k: v.cuda() for k, v in inp.items() if k != "weights"}
    return dev, {k: ([t.cuda() for t in v] if isinstance(v, list) else v.cuda()) for k, v in inp["weights"].items()}


def _whole(inp, pk, pv):
    """The oracle's caches: the prefix's rows, then the request's own."""
    R, d = inp["kv_k"].shape[0], pk.shape[1]
    k, v = (torch.cat([p.expand(R, *p.shape), inp[n]], 1) for p, n in ((pk, "kv_k"), (pv, "kv_v")))
    return _np(k), _np(v), _np(inp["ctx_len"] + pk.shape[0])


def _oracle(cfg, inp, pk, pv, W, seed, offset):
    k, v, n = _whole(inp, pk, pv)
    dims = oc.Dims(n_heads=cfg.n_heads, head_dim=cfg.head_dim, D=1, eps=cfg.eps, rope_base=cfg.rope_base)
    return od.draft_step(_np(inp["parent_hidden"]), _np(inp["frontier"]), _np(inp["pos"]), k, v, n, W, dims, seed, offset)


def _draws(cfg, g, r, seed, offset):
    for rid in range(cfg.R):
        y, m = ov.inverse_cdf(g["q"][rid].astype(np.float64), od.draft_uniform(seed, offset, rid))
        if m > 1e-6:
            assert g["y"][rid] == y
        if r["margin"][rid] > 5e-3:
            assert g["y"][rid] == r["y"][rid]


CASES = [(synth.DRAFT_SMALL, [0, 1, 100, 299, 300]), (synth.DRAFT_SMALL_HD128, [0, 63, 577, 1100])]


@pytest.mark.parametrize("cfg,ctx", CASES)
@pytest.mark.parametrize("group,symmetric", [(128, True), (64, False), (32, False)])
def test_step_with_4bit_maps(cfg, ctx, group, symmetric):
    """Groups that do not divide the small widths (ffn 576, groups of 128) among them."""
    inp, pk, pv = _inputs(cfg, 4, ctx, 0)
    i4 = synth.make_int4_block(inp["weights"], group, symmetric)
    W = oi.draft_weights(oc.weights_to_numpy(inp["weights"]),
                         {k: tuple(None if t is None else (_np(t) if t.dtype != torch.uint8 else t.numpy()) for t in v)
                          for k, v in i4.items()}, group)
    dev, w = _dev(inp)
    step = lib.DraftStep(cfg, w, int4={k: tuple(None if t is None else t.cuda() for t in v) for k, v in i4.items()},
                         int4_group=group)
    h = torch.empty((cfg.R, cfg.d), dtype=torch.bfloat16, device="cuda")
    g = step(**dev, seed=13, offset=3, h_out=h)
    lib.check_errors()
    g = {k: _np(v) for k, v in g.items()}
    r = _oracle(cfg, inp, pk, pv, W, 13, 3)
    check(g, r, list(range(cfg.R)), qbar=Q_BAR)
    _draws(cfg, g, r, 13, 3)


@pytest.mark.parametrize("cfg,ctx", CASES)
@pytest.mark.parametrize("prefix", [1, 127, 700])
def test_step_on_a_shared_prefix(cfg, ctx, prefix):
    inp, pk, pv = _inputs(cfg, 6, ctx, prefix)
    dev, w = _dev(inp)
    step = lib.DraftStep(cfg, w, prefix_len=prefix)
    h = torch.empty((cfg.R, cfg.d), dtype=torch.bfloat16, device="cuda")
    g = step(**dev, seed=8, offset=1, h_out=h, prefix_k=pk.cuda(), prefix_v=pv.cuda())
    lib.check_errors()
    g = {k: _np(v) for k, v in g.items()}
    r = _oracle(cfg, inp, pk, pv, oc.weights_to_numpy(inp["weights"]), 8, 1)
    check(g, r, list(range(cfg.R)), qbar=Q_BAR)
    _draws(cfg, g, r, 8, 1)


def test_serving_round_together():
    """What a serving step runs: a draft round of three with 4-bit maps on a
    shared prompt, the target's attention for the four new tokens of each request,
    its logits to probability rows under penalties and a grammar, verification.
    The round is checked step by step, verification against its oracle, and no
    emitted token is forbidden."""
    cfg, gamma, prefix, seed = synth.DRAFT_SMALL, 3, 260, 31
    R, V = cfg.R, cfg.V
    inp, pk, pv = _inputs(cfg, 9, [0, 1, 100, 290, 297], prefix)
    i4 = synth.make_int4_block(inp["weights"], 64, False)
    W = oi.draft_weights(oc.weights_to_numpy(inp["weights"]),
                         {k: (v[0].numpy(), _np(v[1]), v[2].numpy()) for k, v in i4.items()}, 64)
    dev, w = _dev(inp)
    rnd = lib.DraftRound(cfg, w, gamma, int4={k: tuple(t.cuda() for t in v) for k, v in i4.items()}, int4_group=64,
                         prefix_len=prefix)
    h = torch.empty((R, gamma, cfg.d), dtype=torch.bfloat16, device="cuda")
    pkd, pvd = pk.cuda(), pv.cuda()
    g = rnd(**dev, seed=seed, offset=7, h_out=h, prefix_k=pkd, prefix_v=pvd)
    # the target's attention over the same prompt: grouped heads, the drafts' rows appended
    gen = torch.Generator().manual_seed(2)
    H, Hkv, hd, L = 8, 2, 64, gamma + 1
    rnd_t = lambda *s: torch.randn(s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    att = lib.prefix_attention(rnd_t(R, L, H, hd), rnd_t(prefix, Hkv, hd), rnd_t(prefix, Hkv, hd), rnd_t(R, 310, Hkv, hd),
                               rnd_t(R, 310, Hkv, hd), dev["ctx_len"] + L)
    head = (torch.randn(H * hd, V, generator=gen) * 0.2).cuda()
    logits = att["o"].float().reshape(R, L, H * hd) @ head
    words = np.random.default_rng(3).integers(-2 ** 31, 2 ** 31, (R, L, -(-V // 32))).astype(np.int32)
    mask = torch.from_numpy(words | (words >> 1)).cuda()
    hist = torch.randint(0, V, (R, 50), generator=gen, dtype=torch.int32).cuda()
    rows = lib.logits_probs(logits, hist=hist, draft=g["y"], repetition=torch.full((R,), 1.1, device="cuda"),
                            frequency=torch.full((R,), 0.2, device="cuda"), mask=mask)
    out = lib.spec_verify(rows["p"], g["q"], g["y"], seed, 7)
    lib.check_errors()
    g = {k: _np(v) for k, v in g.items()}
    dims = oc.Dims(n_heads=cfg.n_heads, head_dim=cfg.head_dim, D=1, eps=cfg.eps, rope_base=cfg.rope_base)
    k, v, n = _whole(inp, pk, pv)
    r = od.draft_round(_np(inp["parent_hidden"]), _np(inp["frontier"]), _np(inp["pos"]), k, v, n, W, dims, gamma, seed, 7,
                       forced_y=g["y"], forced_h=g["h"])
    _check_round(cfg, g, r, seed, 7, bar0=Q_BAR)
    assert (rows["status"].cpu().numpy() == 0).all()
    ref = ov.spec_verify(rows["p"].cpu().numpy(), g["q"], g["y"], seed, 7)
    keep = ref["margin"] > 1e-6
    for a, b in (("accepted", "accepted"), ("next_token", "token"), ("n_emit", "n_emit"), ("status", "status")):
        np.testing.assert_array_equal(out[a].cpu().numpy()[keep], ref[b][keep])
    for i in range(R):
        emitted = g["y"][i, :int(out["accepted"][i])].tolist() + [int(out["next_token"][i])]
        for j, t in enumerate(emitted):
            assert (int(mask[i, j, t >> 5]) >> (t & 31)) & 1


def test_round_replayed_from_a_graph():
    cfg = synth.DRAFT_SMALL
    inp, pk, pv = _inputs(cfg, 5, [3, 1, 100, 200, 300], 200)
    i4 = synth.make_int4_block(inp["weights"], 32)
    dev, w = _dev(inp)
    rnd = lib.DraftRound(cfg, w, 2, int4={k: tuple(None if t is None else t.cuda() for t in v) for k, v in i4.items()},
                         int4_group=32, prefix_len=200)
    out = {"q": torch.empty(cfg.R, 2, cfg.V, device="cuda"), "y": torch.empty(cfg.R, 2, dtype=torch.int32, device="cuda")}
    call = lambda: rnd(**dev, seed=1, offset=2, out=out, prefix_k=pk.cuda(), prefix_v=pv.cuda())  # noqa: E731
    pk, pv = pk.cuda(), pv.cuda()
    call()
    want = {k: v.clone() for k, v in out.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for v in out.values():
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["y"], want["y"]) and torch.equal(out["q"], want["q"])
    lib.check_errors()


def test_refusals():
    cfg = synth.DRAFT_SMALL
    inp, pk, pv = _inputs(cfg, 5, [0] * 5, 64)
    dev, w = _dev(inp)
    i4 = {k: tuple(t.cuda() for t in v[:2]) + (None,) for k, v in synth.make_int4_block(inp["weights"], 64).items()}
    f8 = {k: tuple(t.cuda() for t in v) for k, v in synth.make_fp8_block(inp["weights"]).items()}
    with pytest.raises(lib.MtpError):
        lib.DraftStep(cfg, w, fp8=f8, int4=i4)
    with pytest.raises(lib.MtpError):
        lib.DraftStep(cfg, w, int4=i4, int4_group=128)  # scales of groups of 64
    with pytest.raises(lib.MtpError):
        lib.DraftStep(cfg, w, prefix_len=-1)
    with pytest.raises(lib.MtpError):
        lib.DraftStep(cfg, w, int4={**i4, "wq": i4["w_up"]}, int4_group=64)
    step = lib.DraftStep(cfg, w, prefix_len=64)
    for kw in ({}, dict(prefix_k=pk.cuda()), dict(prefix_k=pk.cuda()[:63], prefix_v=pv.cuda()[:63])):
        with pytest.raises(lib.MtpError):
            step(**dev, seed=0, offset=0, **kw)
    with pytest.raises(lib.MtpError):
        lib.DraftStep(cfg, w)(**dev, seed=0, offset=0, prefix_k=pk.cuda(), prefix_v=pv.cuda())
