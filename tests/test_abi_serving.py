"""Host validation of the serving operators' C entries (no launches, no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from deepseek_sequential_mtp_gb300 import build, lib as binding
    build.build()
    return binding.load()


FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)


def test_logits_probs_host_validation(lib):
    from deepseek_sequential_mtp_gb300 import lib as binding

    def call(R=2, L=2, V=100, dtype=0, logits=FAKE, ld=100, p=ctypes.c_void_p(1 << 24), status=None, **prm):
        s = binding.LogitsParams()
        for k, v in prm.items():
            setattr(s, k, v)
        return lib.mtp_logits_probs(R, L, V, dtype, logits, ld, ctypes.byref(s), p, status, None)

    assert call(R=-1) == 1 and call(L=0) == 1 and call(V=0) == 1 and call(dtype=5) == 1
    assert call(R=0, logits=None, p=None) == 0
    assert call(logits=None) == 1 and call(p=None) == 1
    assert call(V=524289, ld=524289) == 7 and call(L=65537) == 7
    assert call(ld=99) == 2
    assert call(logits=ODD) == 3 and call(p=ODD) == 3 and call(status=ODD) == 3 and call(mask=(1 << 20) + 1) == 3
    assert call(dtype=1, logits=ctypes.c_void_p((1 << 20) + 1)) == 3
    assert call(p=FAKE, ld=104) == 1 and call(p=FAKE, dtype=1) == 1  # in place with gaps, or over bf16 logits
    assert call(hist_cap=-1) == 1 and call(n_bias=-1) == 1
    assert call(hist_cap=4) == 1 and call(n_bias=3, bias=1 << 20) == 1
    assert call(hist_cap=262145, hist=1 << 20) == 7 and call(n_bias=4096, bias=1 << 20, bias_ids=1 << 20) == 7
    assert call(R=1 << 20, L=1 << 10) == 7


def test_gemm_int4w_host_validation(lib):
    from deepseek_sequential_mtp_gb300 import lib as binding

    def call(R=4, N=64, K=256, group=128, x=FAKE, q=1 << 20, scale=1 << 20, zero=None, out=FAKE, w=True):
        m = binding.Int4Matrix(q, scale, zero)
        return lib.mtp_gemm_int4w(R, N, K, group, x, ctypes.byref(m) if w else None, out, 0, None)

    assert call(w=False) == 1 and call(x=None) == 1 and call(out=None) == 1 and call(q=None) == 1 and call(scale=None) == 1
    assert call(R=0) == 2 and call(R=33) == 2 and call(N=0) == 2 and call(K=0) == 2
    assert call(K=40) == 3 and call(x=ODD) == 3 and call(q=(1 << 20) + 8) == 3 and call(scale=(1 << 20) + 1) == 3
    assert call(out=ODD) == 3
    assert call(group=48) == 7 and call(group=256) == 7


def test_prefix_attention_host_validation(lib):
    from deepseek_sequential_mtp_gb300 import lib as binding

    def call(q=FAKE, pk=FAKE, pv=FAKE, kk=FAKE, kv=FAKE, ctx=FAKE, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 40, **kw):
        d = binding.PrefixDims(2, 1, 4, 2, 64, 20, 10, 1, 0.0)
        for k, v in kw.items():
            setattr(d, k, v)
        return lib.mtp_prefix_attention(ctypes.byref(d), q, pk, pv, kk, kv, ctx, out, lse, ws, ws_bytes, None)

    assert lib.mtp_prefix_attention(None, *[FAKE] * 9, 1 << 40, None) == 1
    assert call(head_dim=96) == 7
    for bad in (dict(R=0), dict(L=0), dict(n_heads=3), dict(n_kv_heads=0), dict(P=-1), dict(T=-1), dict(R=65536),
                dict(R=1 << 10, L=1 << 10, n_heads=32)):
        assert call(**bad) == 2
        d = binding.PrefixDims(2, 1, 4, 2, 64, 20, 10, 1, 0.0)
        for k, v in bad.items():
            setattr(d, k, v)
        assert lib.mtp_prefix_attention_workspace_bytes(ctypes.byref(d)) == 0
    assert call(scale=-1.0) == 1 and call(scale=float("nan")) == 1
    assert call(q=None) == 1 and call(pk=None) == 1 and call(kv=None) == 1 and call(out=None) == 1 and call(ws=None) == 1
    assert call(q=ODD) == 3 and call(lse=ODD) == 3 and call(ctx=ODD) == 3 and call(q_stride_h=68) == 3
    assert call(kv_stride_t=-8) == 2
    assert call(ws_bytes=64) == 4


def test_draft_round_ext_host_validation(lib):
    from deepseek_sequential_mtp_gb300 import lib as binding, synth
    cfg = synth.DRAFT_SMALL
    dims = binding.Dims(cfg.R, cfg.ctx, cfg.d, cfg.n_heads, cfg.head_dim, cfg.ffn, cfg.V, 1, cfg.eps,
                        cfg.rope_base, binding.MTP_BF16)
    one = (ctypes.c_void_p * 1)(1 << 20)
    w = binding.Weights()
    w.embed = w.head = w.out_norm = 1 << 20
    for k in binding._WEIGHT_LISTS:
        setattr(w, k, ctypes.cast(one, binding._PP))

    def call(ws_bytes=16, **kw):
        ext = binding.DraftExt()
        for k, v in kw.items():
            setattr(ext, k, v)
        return lib.mtp_draft_round_ext(ctypes.byref(dims), ctypes.byref(w), ctypes.byref(ext), *[FAKE] * 6, 1, 0, 0,
                                       FAKE, FAKE, None, FAKE, ws_bytes, None)

    def int4(group=64, q=1 << 20, scale=1 << 20):
        b = binding.BlockInt4()
        b.group = group
        for k in binding.FP8_LINEAR_MAPS:
            setattr(b, k, binding.Int4Matrix(q, scale, None))
        return ctypes.pointer(b)

    assert call() == 4 and call(int4=int4()) == 4 and call(prefix_len=5, prefix_k=1 << 20, prefix_v=1 << 20) == 4
    assert call(prefix_len=-1) == 1 and call(prefix_len=5) == 1 and call(prefix_len=5, prefix_k=1 << 20) == 1
    assert call(prefix_len=5, prefix_k=(1 << 20) + 8, prefix_v=1 << 20) == 3
    assert call(int4=int4(group=16)) == 7 and call(int4=int4(q=None)) == 1 and call(int4=int4(q=(1 << 20) + 4)) == 3
    assert call(int4=int4(scale=(1 << 20) + 1)) == 3
    assert call(int4=int4(), fp8=ctypes.pointer(binding.BlockFp8())) == 1
    size = lambda g, p: lib.mtp_draft_round_ext_workspace_bytes(ctypes.byref(dims), g, p)  # noqa: E731
    assert size(2, 0) == lib.mtp_draft_round_workspace_bytes(ctypes.byref(dims), 2) and size(2, 500) > size(2, 0)
    assert size(0, 0) == 0 and size(32, 0) == 0 and size(1, -1) == 0


def test_logits_probs_refuses_overlapping_rows(lib):
    from deepseek_sequential_mtp_gb300 import lib as binding

    def call(logits, p, dtype=0, ld=100):
        return lib.mtp_logits_probs(2, 3, 100, dtype, ctypes.c_void_p(logits), ld, ctypes.byref(binding.LogitsParams()),
                                    ctypes.c_void_p(p), None, None)

    at, p_bytes = 1 << 20, 6 * 100 * 4
    assert call(at, at + 400) == 1 and call(at, at - 400) == 1      # a row on, a row back
    assert call(at, at + 4 * (5 * 128 + 99), ld=128) == 1           # the last value of the last row
    assert call(at, at - p_bytes + 4, dtype=1) == 1
    assert call(at, at + 600, dtype=1) == 1                         # within the bf16 rows
