"""The serving operators on tensors whose offsets pass 32 bits: rows far apart in memory, and
outputs of more than 2^31 elements.  Samples against fp64."""
import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib
from oracle import prefix as op

pytestmark = pytest.mark.gpu


def _check_attention(got, q, pk, pv, kk, kv, ctx):
    f = [t.detach().cpu().double().numpy() for t in (q, pk, pv, kk, kv)]
    o, lse, mass = op.attention(*f, ctx)
    kmax = max([np.abs(f[i]).max() for i in (1, 3) if f[i].size])
    S = f[0].shape[-1] ** -0.5 * np.abs(f[0]).sum(-1, keepdims=True) * kmax
    go = got["o"].detach().cpu().double().numpy()
    # the bar of test_gpu_prefix_weights.py
    assert (np.abs(go - o) <= 2.0 ** -8 * np.abs(o) + (2.0 ** -15 + 2.0 ** -20 * (S + 4)) * mass + 1e-30).all()


@pytest.mark.parametrize("R,L,H", [(2, 1, 4), (40, 2, 4)])  # few rows, row tiles
def test_caches_that_span_more_than_4_gb(R, L, H):
    """Keys 2^22 elements apart, requests as well: the last rows lie 4.3e9 elements in."""
    P, T, Hkv, hd, far = 1030, 24, 2, 64, 1 << 22
    buf = torch.empty((P, far), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    views = [buf[:, i * 256: i * 256 + Hkv * hd].view(P, Hkv, hd) for i in range(2)]
    own = [buf[P - R * T:, 1024 + i * 256: 1024 + i * 256 + Hkv * hd].unflatten(0, (R, T)).view(R, T, Hkv, hd) for i in range(2)]
    for t in (*views, *own):
        t.copy_(n(*t.shape))
    q = n(R, L, H, hd)
    ctx = [L + (5 * r) % (T - L + 1) for r in range(R)]
    got = lib.prefix_attention(q, views[0], views[1], own[0], own[1], torch.tensor(ctx, dtype=torch.int32, device="cuda"))
    lib.check_errors()
    _check_attention(got, q, *views, *own, ctx)


@pytest.mark.parametrize("R", [1, 32])
def test_4bit_codes_past_4_gb(R):
    N, K = (1 << 20) + 3, 8192  # 4.3e9 bytes of codes; any byte is a pair of them
    q = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    rows = [0, 1, N // 2, N - 2, N - 1]
    g = torch.Generator(device="cuda").manual_seed(2)
    q[rows] = torch.randint(0, 256, (len(rows), K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full((N, K // 128), 0.01, dtype=torch.bfloat16, device="cuda")
    x = torch.randn((R, K), generator=g, device="cuda").to(torch.bfloat16)
    got = lib.gemm_int4w(x, q, s)[:, rows].cpu().double()
    c = torch.stack((q[rows] & 15, q[rows] >> 4), -1).reshape(len(rows), K).cpu().double() - 8
    w = c * s[0, 0].double().item()
    # the bar of test_gpu_int4.py: G/16 + groups + 16 roundings of 2^-23
    bound = 2.0 ** -23 * (8 + K / 128 + 16) * (x.cpu().double().abs() @ w.abs().T)
    assert ((got - x.cpu().double() @ w.T).abs() <= bound).all()


def test_logits_rows_far_apart_and_outputs_past_2_31_elements():
    V, rows = 524288, 4100
    x = torch.empty((rows, 1, V), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    pick = [0, 1, rows // 2, rows - 1]
    x.zero_()
    x[pick] = (torch.randn((len(pick), 1, V), generator=g, device="cuda") * 3).to(torch.bfloat16)
    hist = torch.randint(0, V, (rows, 20), generator=g, device="cuda", dtype=torch.int32)
    rep = torch.full((rows,), 1.5, device="cuda")
    got = lib.logits_probs(x, hist=hist, repetition=rep)
    assert (got["status"] == 0).all()
    for r in pick:
        z = x[r, 0].double()
        u = hist[r].long().unique()
        z[u] = torch.where(z[u] > 0, z[u] / 1.5, z[u] * 1.5)
        p = torch.softmax(z, 0)
        t = -torch.log(p)
        # the bar of test_gpu_logits.py with Z = 30, T = 1
        assert ((got["p"][r, 0].double() - p).abs() <= 2.0 ** -24 * (8 * 30 + 10 * t + 92) * p + 1.2e-38).all()
    del x, got
    far = torch.empty((20, 1 << 28), dtype=torch.bfloat16, device="cuda")
    far[:, :1000] = (torch.randn((20, 1000), generator=g, device="cuda") * 3).to(torch.bfloat16)
    view = far[:, :1000].unsqueeze(1)
    p = lib.logits_probs(view)["p"]
    assert torch.equal(p, lib.logits_probs(view.contiguous())["p"])
