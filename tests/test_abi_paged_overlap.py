"""Outputs of mtp_rope and mtp_kv_append that lie on their inputs, or on themselves, are refused on the host, before anything is
launched (no GPU; what is accepted is tested with tensors, in test_gpu_paged_overlap.py)."""
import ctypes

import pytest

from deepseek_sequential_mtp_gb300 import build, lib as binding

P, Q = 1 << 24, 1 << 28  # addresses that nothing reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("N,H,on,oh", [
    (2, 4, 200, 128), (2, 2, 128, 128), (2, 4, 504, 128), (8, 3, 128, 1016), (7, 8, 1000, 136), (101, 7, 136, 13600), (2, 4, 512, 64),
    (2, 4, 64, 512), (3, 60000, 128, 256), (60000, 3, 256, 128), (4, 4, 384, 256), (2, 3, 0, 127)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rope_rows_on_top_of_one_another(lib, N, H, on, oh, in_place):
    """Refused whichever stride is the smaller one."""
    rot = ctypes.byref(binding.Rotation(P, 64, 0, 1.0))
    x = (Q, on, oh) if in_place else (1 << 50, 0, 0)
    assert lib.mtp_rope(N, H, 128, 1, rot, P, 0, *x, Q, on, oh, None) == 2


def rows(**kw):
    w = binding.KvRows(2, 3, 2, P, P + (1 << 16), Q, Q + (1 << 16))
    w.ctx_len = P
    for k, v in kw.items():
        setattr(w, k, v)
    return ctypes.byref(w)


SIZE = 2 * 3 * 2 * 128 * 2  # bytes of k, v, q and q_out


@pytest.mark.parametrize("bad", [
    dict(q_out=P), dict(q_out=P + SIZE - 16), dict(q_out=P + (1 << 16) - SIZE + 16), dict(q_out=P + (1 << 16)),   # k, v
    dict(q_out=Q + 16), dict(q_out=Q - SIZE + 16), dict(q_out=Q + SIZE - 16),                                       # part of q
    dict(k=Q, v=Q, q_out=Q),                                                                                        # q in place, and it is k
    dict(q_stride_h=256, q_stride_t=768, q_out=Q + SIZE),                                                           # among rows of q
    dict(kv_stride_h=256, kv_stride_t=768, q_out=P + SIZE)])
def test_append_refuses_queries_over_inputs(lib, bad):
    c = binding.PagedCache(P, P, P, P, P, 8, 64, 4, 2, 128, binding.MTP_E4M3)
    assert lib.mtp_kv_append(ctypes.byref(c), rows(**bad), None, None) == 1
