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
from oracle import paged
from test_gpu_paged_attention import case, check, values

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


def check_all(c, table, q, ctx, got, n_new=None, causal=True, rows=None):
    """check, and lse is NaN where the oracle's is and nowhere else (check passes a NaN over)."""
    check(c, table, q, ctx, got, n_new, causal, rows=rows)
    R, L, H, hd = q.shape
    rows = list(range(R)) if rows is None else rows
    cap = table.shape[1] * c["k_pages"].shape[2]
    new = None if n_new is None else [max(0, min(int(n_new[r]), L)) for r in rows]
    with np.errstate(invalid="ignore"):
        lse = paged.attention(q[rows].double().numpy(), values(c, "k"), values(c, "v"), table.numpy()[rows],
                              [max(0, min(int(ctx[r]), cap)) for r in rows], new, causal)[1]
    np.testing.assert_array_equal(np.isnan(got["lse"][rows].cpu().numpy()), np.isnan(lse))


@types
@forms
def test_bad_pages_are_passed_over(kernel, L, G, eight):
    """Pages out of range set the error and are not read, at a request's beginning, within it, at its end, and within a block of
    128 keys of which others are good; the requests that name none have their outputs."""
    c, table, q = case(5, L, 2 * G, 2, 64, 16, 12, eight, L + G + 1)
    ctx, n = [192, 140, 190, 133, 64], c["k_pages"].shape[0]
    bad = table.clone()
    bad[0, 3], bad[2, 0], bad[2, 1], bad[3, 8] = n, -7, 2147483647, -2147483648
    got = call(kernel, c, bad, q, ctx, errors=True, causal=False)
    check_all(c, table, q, ctx, got, causal=False, rows=[1, 4])
    if kernel != "dense":  # (whose gathered rows are zeros there)
        for r, skip in ((0, [3]), (2, [0, 1]), (3, [8])):
            keep = [i for i in range(12) if i not in skip] + skip
            left = sum(max(0, min(16, ctx[r] - 16 * i)) for i in range(12) if i not in skip)
            one = {k: v[r:r + 1] for k, v in got.items()}
            check_all(c, table[r:r + 1, keep].contiguous(), q[r:r + 1], [left], one, causal=False)
    again = call(kernel, c, table, q, ctx)  # and what follows is as ever
    check_all(c, table, q, ctx, again)


@types
@pytest.mark.parametrize("kernel,L,G", FORMS[:-1])  # (tables of more than 4 GB: the kernels of `long`)
@pytest.mark.parametrize("causal", [True, False])
def test_lengths_beyond_the_table_and_below_zero(kernel, L, G, eight, causal):
    """Lengths as the device holds them: clamped to the table's rows, which are all written here, and to zero."""
    per = 66 if kernel == "long" else 8
    c, table, q = case(5, L, 2 * G, 2, 64, 16, per, eight, L + G + 2)
    ctx = [16 * per + 1, 2147483647, -1, -2147483648, 16 * per]
    got = call(kernel, c, table, q, ctx, causal=causal)
    check_all(c, table, q, ctx, got, causal=causal)
    new = [L, 0, L, L, 2147483647]
    check_all(c, table, q, ctx, call(kernel, c, table, q, ctx, new, causal=causal), new, causal=causal)


@types
@forms
@pytest.mark.parametrize("hd,page", [(64, 48), (128, 80), (64, 96), (128, 192), (64, 144), (128, 1008)])
def test_pages_that_are_no_power_of_two(kernel, L, G, eight, hd, page):
    per = max(1, 400 // page)
    c, table, q = case(3, L, 2 * G, 2, hd, page, per, eight, page + L)
    ctx = [page * per, page * per - 7, min(page * per, page + 1)]
    check_all(c, table, q, ctx, call(kernel, c, table, q, ctx))


@types
@forms
def test_fewer_rows_than_new_tokens(kernel, L, G, eight):
    """Causal: the tokens before a request's first row see nothing."""
    c, table, q = case(6, L, 2 * G, 2, 64, 16, 8, eight, L + G + 3)
    ctx = [0, 1, L - 1, L, L + 1, 128]
    check_all(c, table, q, ctx, call(kernel, c, table, q, ctx))
    new = [L, L - 1, max(1, L // 2), 1, L, 0]
    check_all(c, table, q, ctx, call(kernel, c, table, q, ctx, new), new)


@pytest.mark.parametrize("name", ["k", "v"])
@types
@forms
def test_not_finite_where_seen(kernel, L, G, eight, name):
    """NaN, and in bf16 both infinities: a value that a token sees makes its outputs of that dimension not finite; a key gives the score that it
    gives in the oracle; what a token does not see is nothing to it."""
    R, ctx = 4, [140, 140, 140, 140]
    c, table, q = case(R, L, 2 * G, 2, 64, 16, 10, eight, L + G + 4)
    kinds = [0x7F, 0xFF] if eight else [float("nan"), float("inf"), float("-inf")]
    pages = c[name + "_pages"]

    def put(r, j, value, d):
        pages[int(table[r, j // 16]), :, j % 16, d] = value
    for r in range(R):
        for j in range(140, 160):  # behind the rows
            for d in range(64):
                put(r, j, kinds[(r + d) % len(kinds)], d)
    for i, v in enumerate(kinds):
        put(1, 139, v, 3 * i)           # of the last token
        put(2, 3, v, 3 * i + 1)         # at the beginning: all see it
        put(3, 140 - L, v, 3 * i + 2)   # of the first token: all see it
        put(3, 140 - (L + 1) // 2, v, 30 + i)
    got = call(kernel, c, table, q, ctx)
    plain = {k: v.clone() for k, v in c.items()}
    if not eight and name == "v":
        plain["v_pages"][torch.isinf(pages)] = float("nan")
        got["o"] = torch.where(torch.isinf(got["o"]), torch.nan, got["o"])
    check_all(plain, table, q, ctx, got)


@types
@pytest.mark.parametrize("G,L", [(1, 2), (8, 5), (2, 40)])
def test_offsets_past_32_bits(eight, G, L):
    """Pages beyond 2^32 bytes under tables that take the kernels for long ones, and gathered rows."""
    hd, page, Hkv, per = 128, 256, 4, 5
    n = (1 << 32) // (page * Hkv * hd) + 9
    c, table, q = case(1, L, Hkv * G, Hkv, hd, page, per, eight, G)
    d = {k: torch.zeros((n, *v.shape[1:]), dtype=v.dtype, device="cuda") for k, v in c.items()}
    place = torch.tensor([n - 1, n - 3, 1, n - 2, n - 4, n - 6])
    for k, v in c.items():
        d[k][place.cuda()] = v.cuda()
    assert n * page * Hkv * hd * (1 if eight else 2) > 1 << 32 and per * page > 1024
    got = lib.paged_attention(q.cuda(), **d, page_table=place[table.long()].int().cuda(),
                              ctx_len=torch.tensor([1200], dtype=torch.int32).cuda())
    lib.check_errors()
    check_all(c, table, q, [1200], got)


@types
@pytest.mark.parametrize("L,G", [(1, 2), (2, 8)])
def test_long_contexts(eight, L, G):
    """70000 rows, most of which have weights far below the largest."""
    c, table, q = case(2, L, G, 1, 64, 256, 274, eight, 5)
    ctx = [70000, 69999]
    check_all(c, table, q, ctx, call("long", c, table, q, ctx))
