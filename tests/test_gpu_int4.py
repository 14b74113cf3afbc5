"""mtp_gemm_int4w on the GPU against the exact dequantisation in fp64.

Tolerance of an entry (derived): products of bf16 activations and integer
codes are exact; a tensor-core step sums 16 of them with the accumulator to
within 2^-23 of the largest partial (truncation), a group is G/16 such steps,
the scaled groups are added by fused multiply-adds (2^-24 each, at most
`groups` of them over the k-warps and the cluster, plus 16 for the joins):
  2^-23 (G/16 + groups + 16) Σ_k |x||W|, and as much again of the old value
when it is added to."""
import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib
from oracle import int4 as oi

pytestmark = pytest.mark.gpu


def _case(R, N, K, group, zero, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    groups = -(-K // group)
    s = ((torch.rand((N, groups), generator=g) + 0.2) * 0.01 * torch.sign(torch.randn((N, groups), generator=g))).to(torch.bfloat16)
    z = torch.randint(0, 16, (N, groups), generator=g, dtype=torch.uint8) if zero else None
    x = (torch.randn((R, K), generator=g) * torch.exp(torch.randn((R, K), generator=g))).to(torch.bfloat16)
    return x, q, s, z


def _bound(x, W, group):
    K = x.shape[1]
    return 2.0 ** -23 * (group / 16 + -(-K // group) + 16) * (np.abs(x) @ np.abs(W).T)


def _dev(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("R,N,K", [(1, 1, 32), (1, 2816, 1024), (2, 17, 96), (3, 40, 416), (4, 100, 1120), (8, 129, 288),
                                   (9, 300, 2048), (16, 257, 544), (17, 96, 1312), (31, 1000, 192), (32, 130, 4128),
                                   (5, 1003, 2848), (32, 512, 18432)])
def test_gemm_parity(R, N, K, group):
    zero = (R + N) % 2 == 0
    x, q, s, z = _case(R, N, K, group, zero, R * 1000 + N + K)
    out = lib.gemm_int4w(*_dev(x, q, s, z), group=group)
    torch.cuda.synchronize()
    xd = x.double().numpy()
    W = oi.dequantize(q.numpy(), s.double().numpy(), None if z is None else z.numpy(), group)
    assert (np.abs(out.cpu().double().numpy() - xd @ W.T) <= _bound(xd, W, group) + 1e-30).all()


def test_accumulate_and_repeatability():
    x, q, s, z = _case(7, 500, 3008, 64, True, 5)
    old = torch.randn(7, 500, generator=torch.Generator().manual_seed(1))
    d = _dev(x, q, s, z)
    plain = lib.gemm_int4w(*d, group=64)
    out = old.cuda()
    got = lib.gemm_int4w(*d, group=64, out=out, accumulate=True)
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, old.cuda() + plain)
    for _ in range(10):
        assert torch.equal(lib.gemm_int4w(*d, group=64), plain)


def test_tokens_do_not_touch_each_other():
    """NaN and infinities in one token stay in its row; weights of codes equal
    to their zero point times an infinity are NaN, as the product says."""
    x, q, s, _ = _case(6, 64, 256, 128, False, 9)
    want = lib.gemm_int4w(*_dev(x, q, s), group=128)
    x[2, 5], x[4, 200] = float("nan"), float("inf")
    got = lib.gemm_int4w(*_dev(x, q, s), group=128)
    keep = [0, 1, 3, 5]
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[2]).all() and not torch.isfinite(got[4]).any()


def test_rows_behind_and_beside_stay():
    """A matrix whose rows end inside a tile writes only its own columns."""
    x, q, s, z = _case(3, 50, 512, 32, True, 2)
    buf = torch.full((3 * 50 + 64,), 7.0, device="cuda")
    out = buf[:150].view(3, 50)
    lib.gemm_int4w(*_dev(x, q, s, z), group=32, out=out)
    assert (buf[150:] == 7.0).all() and not (out == 7.0).any()


def test_streams_and_graph():
    x, q, s, z = _case(4, 300, 2048, 128, True, 3)
    d = _dev(x, q, s, z)
    want = lib.gemm_int4w(*d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.gemm_int4w(*d, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = lib.gemm_int4w(*d)
    d[0].mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 2 * want)  # a power of two scales every exact step


def test_refusals():
    x, q, s, z = _dev(*_case(4, 64, 256, 128, True, 4))
    for args, kw in (((x[:, :128].contiguous(), q, s, z), {}), ((x, q, s[:, :1], z), {}), ((x, q, s.float(), z), {}),
                     ((x, q, s, z.int()), {}), ((x, q, s, z), dict(group=48)), ((x, q, s, z), dict(group=0)),
                     ((x, q, s, z), dict(group=64)), ((x.float(), q, s, z), {}), ((x, q, s, z), dict(accumulate=True)),
                     ((x, q, s, z), dict(out=torch.zeros(4, 63, device="cuda"))), ((x.cpu(), q, s, z), {}),
                     ((torch.zeros(33, 256, dtype=torch.bfloat16, device="cuda"), q, s, z), {}),
                     ((torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda"), q, s, z), {}),
                     ((x[:, :248].contiguous(), q[:, :124].contiguous(), s, z), {}), ((x.t(), q, s, z), {})):
        with pytest.raises(lib.MtpError):
            lib.gemm_int4w(*args, **kw)


@pytest.mark.parametrize("R", [18, 23, 24, 25])
def test_tiles_of_tokens(R):
    """Token counts around the borders of the tiles of 8, long enough for a split of k."""
    for group, N, K in ((128, 700, 7168), (32, 130, 2080)):
        x, q, s, z = _case(R, N, K, group, R % 2 == 0, 50 * R + group)
        out = lib.gemm_int4w(*_dev(x, q, s, z), group=group)
        torch.cuda.synchronize()
        xd = x.double().numpy()
        W = oi.dequantize(q.numpy(), s.double().numpy(), None if z is None else z.numpy(), group)
        assert (np.abs(out.cpu().double().numpy() - xd @ W.T) <= _bound(xd, W, group) + 1e-30).all()
