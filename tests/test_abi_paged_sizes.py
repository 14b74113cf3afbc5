"""mtp_kv_append, mtp_kv_gather at the ends of their sizes (no GPU: nothing is launched)."""
import ctypes

import pytest

from deepseek_sequential_mtp_gb300 import build, lib as binding

P = 1 << 20  # an address that nothing reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def cache(**kw):
    c = binding.PagedCache(P, P, P, P, P, 8, 64, 4, 2, 128, binding.MTP_E4M3)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def rows(R, L, **kw):
    w = binding.KvRows(R, L, 0, P, P)
    w.ctx_len = P
    for k, v in kw.items():
        setattr(w, k, v)
    return ctypes.byref(w)


@pytest.mark.parametrize("L", [2147483647, 2147483634, 2147483633])
def test_more_blocks_than_a_launch_has(lib, L):
    """17 requests of that many rows: more CTAs than a grid holds, counted without passing 31 bits on the way."""
    assert lib.mtp_kv_append(cache(), rows(17, L), None, None) == 7


def test_a_batch_without_requests(lib):
    """Its page table is an empty tensor, whose address is null."""
    none = cache(page_table=None)
    assert lib.mtp_kv_append(none, rows(0, 4), None, None) == 0
    assert lib.mtp_kv_append(none, rows(0, 4, k=None, v=None, ctx_len=None), None, None) == 0
    assert lib.mtp_kv_gather(none, 0, 16, None, None, None, None) == 0
    for bad in (dict(page=24), dict(dtype=0), dict(head_dim=96)):  # what does not depend on the batch is still checked
        assert lib.mtp_kv_append(cache(**bad), rows(0, 4), None, None) == 7
        assert lib.mtp_kv_gather(cache(**bad), 0, 16, None, None, None, None) == 7
    assert lib.mtp_kv_append(none, rows(2, 4), None, None) == 1
    assert lib.mtp_kv_gather(none, 2, 16, P, P, P, None) == 1
