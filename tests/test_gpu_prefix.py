"""mtp_prefix_attention on the GPU against the fp64 oracle.

Tolerances (derived).  A softmax weight enters the product with the values as
bf16, off by at most 2^-8 of itself, so the output moves by at most 2^-8 A,
A = Σ p |v| / Σ p; the output's own rounding to bf16 is 2^-8 |o| at most.  The
scores are fp32 sums of exact products, off by 2^-23 per 16-wide step of the sum
S = scale Σ |q k|, which moves a weight by that factor: hd/16 + 4 steps, with the
exponential's 2^-22, far below the rest: 2^-20 (S + 4) A covers them.
lse moves by the scores' error and a few roundings of its own value:
2^-22 (hd/8 S + 8 + 4 |lse|)."""
import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib
from oracle import prefix as op

pytestmark = pytest.mark.gpu


def _inputs(R, L, H, Hkv, hd, P, T, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    return dict(q=(torch.randn((R, L, H, hd), generator=g) * std).to(torch.bfloat16), prefix_k=n(P, Hkv, hd),
                prefix_v=n(P, Hkv, hd), kv_k=n(R, T, Hkv, hd), kv_v=n(R, T, Hkv, hd))


def _np(t):
    return t.detach().cpu().double().numpy()


def _check(a, ctx, got, causal=True, scale=None, rows=None):
    """Compares the requests `rows` (all)."""
    rows = list(range(a["q"].shape[0])) if rows is None else rows
    f = {k: _np(v[rows] if k in ("q", "kv_k", "kv_v") else v) for k, v in a.items()}
    ctx = [int(ctx[r]) for r in rows]
    for k in ("kv_k", "kv_v"):  # what is past ctx_len is not looked at
        f[k] = np.where(np.arange(f[k].shape[1])[None, :, None, None] < np.array(ctx)[:, None, None, None], f[k], 0.0)
    o, lse, mass = op.attention(f["q"], f["prefix_k"], f["prefix_v"], f["kv_k"], f["kv_v"], ctx, causal, scale)
    hd = f["q"].shape[-1]
    sc = hd ** -0.5 if scale is None else scale
    kmax = max([np.abs(f[k]).max() for k in ("prefix_k", "kv_k") if f[k].size] + [0.0])
    S = sc * np.abs(f["q"]).sum(-1, keepdims=True) * kmax
    go, gl = _np(got["o"][rows]), _np(got["lse"][rows])
    assert np.isfinite(go).all()
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -20 * (S + 4)) * mass + 1e-30
    bad = np.abs(go - o) - bound
    assert (bad <= 0).all(), (bad.max(), np.unravel_index(bad.argmax(), bad.shape))
    empty = np.isneginf(lse)
    np.testing.assert_array_equal(np.isneginf(gl), empty)
    assert (go[empty] == 0).all()
    with np.errstate(invalid="ignore"):
        err = np.abs(np.where(empty, 0, gl - lse))
    assert (err <= 2.0 ** -22 * (hd / 8 * S[..., 0] + 8 + 4 * np.abs(np.where(empty, 0, lse)))).all()


def _run(a, ctx, **kw):
    got = lib.prefix_attention(**{k: v.cuda() for k, v in a.items()},
                               ctx_len=None if ctx is None else torch.tensor(ctx, dtype=torch.int32).cuda(), **kw)
    lib.check_errors()
    return got


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("R,L,H,Hkv,P,T,ctx", [
    (1, 1, 1, 1, 1, 0, [0]),                       # one key
    (1, 1, 1, 1, 0, 1, [1]),
    (2, 1, 2, 2, 128, 128, [128, 1]),              # whole blocks, one row
    (3, 2, 4, 2, 127, 130, [2, 129, 130]),         # ragged, grouped heads, causal inside a block
    (4, 1, 2, 1, 300, 64, [0, 1, 63, 64]),         # an empty own cache beside others
    (2, 5, 8, 1, 40, 300, [5, 131]),               # 40 rows per own item, causal across blocks
    (40, 5, 4, 2, 700, 20, None),                  # 400 rows per key head: pairs of tiles and a single one
    (30, 5, 2, 2, 260, 5, None),                   # 150 rows: a pair whose second tile is ragged
    (2, 70, 4, 1, 200, 400, [70, 333]),            # 280 rows in an own item, causal over two tiles
    (5, 3, 3, 3, 0, 500, [0, 3, 2, 499, 500]),     # no prefix; fewer rows than new tokens
    (3, 1, 2, 2, 5000, 0, None),                   # no own caches
])
def test_shapes(hd, R, L, H, Hkv, P, T, ctx):
    a = _inputs(R, L, H, Hkv, hd, P, T, R + L + P + T)
    if ctx is None and T > 0:
        ctx = [min(T, L + r % (T - L + 1)) for r in range(R)]
    _check(a, ctx if ctx else [0] * R, _run(a, ctx))


@pytest.mark.parametrize("causal,scale", [(False, None), (True, 0.3), (False, 0.01)])
def test_causal_flag_and_scale(causal, scale):
    a = _inputs(3, 4, 4, 2, 64, 150, 200, 3)
    _check(a, [2, 130, 200], _run(a, [2, 130, 200], causal=causal, scale=scale), causal, scale)


def test_large_scores_move_the_maximum():
    """Scores in the hundreds that grow along the keys: the running maximum is
    replaced in block after block."""
    a = _inputs(2, 2, 2, 1, 128, 1500, 300, 4, std=4.0)
    ramp = torch.linspace(0.2, 6.0, 1500)[:, None, None]
    a["prefix_k"] = (a["prefix_k"].float() * ramp).to(torch.bfloat16)
    _check(a, [300, 7], _run(a, [300, 7]))


def test_rows_past_the_length_hold_anything():
    """NaN and infinities behind ctx_len, in keys and in values, change nothing."""
    for L in (2, 80):
        a = _inputs(3, L, 2, 1, 64, 100, 310, 5)
        ctx = [L, 129 + L, 300]
        want = _run(a, ctx)
        for r in range(3):
            a["kv_k"][r, ctx[r]:] = float("nan")
            a["kv_v"][r, ctx[r]:] = float("nan")
            a["kv_v"][r, min(ctx[r] + 1, 309):] = float("inf")
        got = _run(a, ctx)
        assert torch.equal(got["o"], want["o"]) and torch.equal(got["lse"], want["lse"])
    _check(a, ctx, got)


def test_lengths_are_clamped():
    a = _inputs(2, 1, 2, 2, 64, 10, 30, 6)
    got, want = _run(a, [-5, 99]), _run(a, [0, 30])
    assert torch.equal(got["o"], want["o"])


def test_strides_and_head_orders():
    """Heads before tokens, rows inside a wider fused tensor, a prefix that is a
    slice of one request's cache."""
    R, L, H, Hkv, hd, P, T = 3, 2, 4, 2, 64, 200, 150
    a = {k: v.cuda() for k, v in _inputs(R, L, H, Hkv, hd, P, T, 7).items()}
    ctx = torch.tensor([2, 100, 150], dtype=torch.int32, device="cuda")
    want = lib.prefix_attention(**a, ctx_len=ctx)
    b = dict(a)
    b["q"] = a["q"].permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    for k in ("prefix_k", "prefix_v"):
        b[k] = a[k].transpose(0, 1).contiguous().transpose(0, 1)
    fused = torch.zeros(R, T, Hkv, 3, hd, dtype=torch.bfloat16, device="cuda")
    fused[:, :, :, 0], fused[:, :, :, 2] = a["kv_k"], a["kv_v"]
    b["kv_k"], b["kv_v"] = fused[:, :, :, 0], fused[:, :, :, 2]
    got = lib.prefix_attention(**b, ctx_len=ctx)
    assert torch.equal(got["o"], want["o"]) and torch.equal(got["lse"], want["lse"])
    c = dict(a)
    c["prefix_k"], c["prefix_v"] = a["kv_k"][1, 10:90], a["kv_v"][1, 10:90]
    _check({k: v.cpu() for k, v in c.items()}, ctx.tolist(), lib.prefix_attention(**c, ctx_len=ctx))


def test_sharing_changes_nothing():
    """A batch on a shared prefix equals each request with the prefix copied into
    its own cache, to the rounding of the weights."""
    R, H, hd, P, T = 6, 4, 128, 384, 64
    a = {k: v.cuda() for k, v in _inputs(R, 1, H, H, hd, P, T, 8).items()}
    ctx = torch.tensor([1, 10, 33, 64, 2, 50], dtype=torch.int32, device="cuda")
    got = lib.prefix_attention(**a, ctx_len=ctx)
    own = {k: torch.cat([a["prefix" + k[2:]].expand(R, P, H, hd), a[k]], 1).contiguous() for k in ("kv_k", "kv_v")}
    none = a["prefix_k"][:0]
    alone = lib.prefix_attention(a["q"], none, none, own["kv_k"], own["kv_v"], ctx + P)
    lib.check_errors()
    assert torch.allclose(got["lse"], alone["lse"], rtol=0, atol=1e-4)
    assert (got["o"].float() - alone["o"].float()).abs().max() < 2.0 ** -6


def test_large_batches_and_long_prefixes_on_samples():
    """The sizes that the operator is for, a few requests against the oracle."""
    for R, L, H, Hkv, hd, P, T, rows in ((32, 5, 32, 8, 128, 8192, 512, [0, 31]), (32, 1, 56, 56, 128, 8192, 256, [17]),
                                         (2, 1, 16, 2, 64, 65001, 100, [1]), (600, 1, 2, 1, 64, 513, 40, [0, 300, 599])):
        a = _inputs(R, L, H, Hkv, hd, P, T, P + R)
        ctx = [L + (37 * r) % (T - L + 1) for r in range(R)]
        _check(a, ctx, _run(a, ctx), rows=rows)


def test_same_bits_streams_and_graphs():
    a = {k: v.cuda() for k, v in _inputs(5, 2, 4, 2, 128, 900, 200, 9).items()}
    ctx = torch.tensor([2, 200, 77, 129, 128], dtype=torch.int32, device="cuda")
    want = lib.prefix_attention(**a, ctx_len=ctx)
    for _ in range(5):
        assert torch.equal(lib.prefix_attention(**a, ctx_len=ctx)["o"], want["o"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.prefix_attention(**a, ctx_len=ctx, stream=side)
    side.synchronize()
    assert torch.equal(got["o"], want["o"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = lib.prefix_attention(**a, ctx_len=ctx)
    ctx.copy_(torch.tensor([3, 50, 200, 2, 5], dtype=torch.int32))  # lengths may change between replays
    a["q"].mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    want = lib.prefix_attention(**a, ctx_len=ctx)
    assert torch.equal(out["o"], want["o"]) and torch.equal(out["lse"], want["lse"])
    lib.check_errors()


def test_refusals():
    a = {k: v.cuda() for k, v in _inputs(2, 1, 4, 2, 64, 20, 10, 1).items()}
    ctx = torch.ones(2, dtype=torch.int32, device="cuda")
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    for kw in (dict(q=a["q"].float()), dict(q=a["q"][0]), dict(q=z(2, 1, 3, 64)), dict(q=z(2, 1, 4, 32)), dict(q=z(0, 1, 4, 64)),
               dict(prefix_v=z(21, 2, 64)), dict(prefix_k=z(20, 2, 128), prefix_v=z(20, 2, 128)),
               dict(prefix_k=a["prefix_k"][:, :1].expand(20, 2, 64), prefix_v=a["prefix_v"][:, :1].expand(20, 2, 64)),
               dict(kv_v=None), dict(kv_k=z(3, 10, 2, 64), kv_v=z(3, 10, 2, 64)), dict(ctx_len=ctx.long()),
               dict(ctx_len=torch.ones(3, dtype=torch.int32, device="cuda")), dict(scale=-1.0), dict(scale=float("nan")),
               dict(kv_k=None, kv_v=None), dict(ws=torch.zeros(16, dtype=torch.uint8, device="cuda")),
               dict(q=a["q"].cpu()), dict(q=z(2, 1, 4, 68)[..., :64])):
        with pytest.raises(lib.MtpError):
            lib.prefix_attention(**{**a, "ctx_len": ctx, **kw})


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("R,L,H,Hkv,P,T,ctx", [
    (8, 1, 4, 2, 1000, 65, [1, 16, 17, 32, 33, 63, 64, 65]),   # 16 rows on the prefix, every tail of a block
    (17, 1, 2, 2, 300, 40, None),                  # 17 rows: the prefix on row tiles, the own caches not
    (3, 16, 2, 2, 50, 700, [16, 31, 700]),         # 16 rows per own item, many blocks
    (3, 17, 2, 2, 50, 700, [17, 300, 699]),        # 17: two tiles of 16 rows
    (2, 8, 8, 2, 0, 400, [8, 400]),                # 32 rows, no prefix
    (2, 11, 6, 2, 0, 400, [12, 399]),              # 33 rows
    (1, 1, 3, 1, 20000, 3000, [2999]),             # one request over all CTAs
    (150, 1, 2, 1, 64, 200, None),                 # more requests than lanes, items cut anywhere
    (1, 32, 1, 1, 0, 33, [20]),                    # fewer own rows than new tokens
])
def test_few_rows(hd, R, L, H, Hkv, P, T, ctx):
    a = _inputs(R, L, H, Hkv, hd, P, T, 7 * R + L + P + T)
    if ctx is None:
        ctx = [0 if r % 11 == 5 else 1 + (53 * r) % T for r in range(R)]
    _check(a, ctx, _run(a, ctx))


def test_few_rows_past_the_length_hold_anything():
    for L, H in ((1, 2), (5, 8), (16, 4)):  # 1, 20 and 32 rows per own item
        a = _inputs(3, L, H, 2, 128, 100, 310, 15)
        ctx = [L, 129 + L, 300]
        want = _run(a, ctx)
        for r in range(3):
            a["kv_k"][r, ctx[r]:] = float("inf")
            a["kv_v"][r, ctx[r]:] = float("nan")
        got = _run(a, ctx)
        assert torch.equal(got["o"], want["o"]) and torch.equal(got["lse"], want["lse"])


def test_no_wait_runs_out():
    """A wait that runs into its limit takes more than a second; these calls take
    some 0.1 ms, on every kernel and with rings that are filled many times."""
    for R, L, H, Hkv, P, T in ((32, 1, 56, 56, 8192, 256), (4, 1, 8, 8, 20000, 3000), (8, 5, 16, 4, 0, 3000), (3, 20, 16, 4, 4000, 900)):
        a = {k: v.cuda() for k, v in _inputs(R, L, H, Hkv, 128, P, T, 16).items()}
        lib.prefix_attention(**a)
        torch.cuda.synchronize()
        t0, t1 = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        t0.record()
        lib.prefix_attention(**a)
        t1.record()
        torch.cuda.synchronize()
        assert t0.elapsed_time(t1) < 100, t0.elapsed_time(t1)
    lib.check_errors()


def test_two_calls_at_once():
    """Calls of both kernels side by side on two streams, each with its own workspace."""
    a = {k: v.cuda() for k, v in _inputs(6, 2, 8, 4, 128, 3000, 500, 17).items()}
    b = {k: v.cuda() for k, v in _inputs(24, 5, 8, 2, 128, 2000, 300, 18).items()}
    want = [lib.prefix_attention(**x) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(6):
        for i, x in enumerate((a, b)):
            got[i].append(lib.prefix_attention(**x, stream=streams[i]))
    torch.cuda.synchronize()
    lib.check_errors()
    for i in range(2):
        for g in got[i]:
            assert torch.equal(g["o"], want[i]["o"]) and torch.equal(g["lse"], want[i]["lse"])
