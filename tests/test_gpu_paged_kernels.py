"""mtp_paged_attention: what every kernel behind it has to hold, with the kernel that a call takes made sure of.

  item   short tables (no workspace)
  long   tables for more: the kernel of 8 bits, or that of bf16
  dense  64 rows per key head and more: gathered rows
  tiles  the same under a table whose copy would be above 4 GB: the kernels of `long`, tile by tile
"""
import ctypes

import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib
from test_gpu_paged_attention import case, check

pytestmark = pytest.mark.gpu
# kernel, new tokens, query heads per key head
FORMS = [("item", 1, 1), ("item", 5, 8), ("long", 1, 1), ("long", 1, 8), ("long", 3, 8), ("long", 5, 8), ("dense", 70, 1), ("dense", 9, 8),
         ("tiles", 70, 1)]
forms = pytest.mark.parametrize("kernel,L,G", FORMS)
types = pytest.mark.parametrize("eight", [True, False])


def workspace(d, table, R, L, H):
    k = d["k_pages"]
    eight = k.dtype == torch.uint8
    c = lib.PagedCache(None, None, None, None, None, k.shape[0], k.shape[2], table.shape[1], k.shape[1], k.shape[3],
                       lib.MTP_E4M3 if eight else lib.MTP_BF16)
    return lib.load().mtp_paged_attention_workspace_bytes(ctypes.byref(lib.PagedDims(R, L, H, 1)), ctypes.byref(c))


def call(kernel, c, table, q, ctx, n_new=None, errors=0, **kw):
    """One call with the table widened (by places that nothing looks at) to what takes the kernel."""
    R, L, H, hd = q.shape
    page, Hkv = c["k_pages"].shape[2], c["k_pages"].shape[1]
    rows = {"item": 0, "long": 1040, "dense": 0, "tiles": (1 << 31) // (2 * R * Hkv * hd) + page}[kernel]
    more = max(0, -(-rows // page) - table.shape[1])
    wide = torch.cat([table, torch.full((R, more), -1, dtype=torch.int32)], 1)
    d = {k: v.cuda() for k, v in c.items()}
    size, copy = workspace(d, wide, R, L, H), 4 * R * wide.shape[1] * page * Hkv * hd
    assert (size == 0) == (kernel == "item") and (L * (H // Hkv) >= 64) == (kernel in ("dense", "tiles"))
    assert kernel not in ("dense", "tiles") or (size > copy) == (kernel == "dense")
    got = lib.paged_attention(q.cuda(), **d, page_table=wide.cuda(), ctx_len=torch.tensor(ctx, dtype=torch.int32).cuda(),
                              n_new=None if n_new is None else torch.tensor(n_new, dtype=torch.int32).cuda(), **kw)
    if errors:
        with pytest.raises(lib.MtpError, match=hex(0x10008 if kernel == "dense" else 0x20008)):
            lib.check_errors()
    else:
        lib.check_errors()
    return got


@types
@forms
@pytest.mark.parametrize("causal", [True, False])
def test_a_request_that_sits_out_is_not_looked_at(kernel, L, G, eight, causal):
    """Its table may hold anything, whatever its length: no error, zeros, and the others' outputs are theirs."""
    c, table, q = case(3, L, 2 * G, 2, 64, 16, 8, eight, L + G)
    ctx, new = [128, 100, 77], [L, 0, max(1, L - 1)]
    table[1] = torch.tensor([-1, 2147483647, c["k_pages"].shape[0], -5, -1, -1, -1, -1], dtype=torch.int32)
    got = call(kernel, c, table, q, ctx, new, causal=causal)
    assert (got["o"][1] == 0).all() and torch.isneginf(got["lse"][1]).all()
    check(c, table, q, ctx, got, new, causal=causal, rows=[0, 2])
