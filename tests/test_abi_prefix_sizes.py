"""A draft round's prefix that the attention over it does not take is refused on the host,
before anything is launched (no GPU)."""
import ctypes

from deepseek_sequential_mtp_gb300 import build, lib as binding, synth


def test_prefix_lengths_beyond_the_attention():
    build.build()
    lib = binding.load()
    cfg = synth.DRAFT_SMALL
    fake = ctypes.c_void_p(1 << 20)
    one = (ctypes.c_void_p * 1)(1 << 20)
    w = binding.Weights()
    w.embed = w.head = w.out_norm = 1 << 20
    for k in binding._WEIGHT_LISTS:
        setattr(w, k, ctypes.cast(one, binding._PP))

    def dims(ctx):
        return binding.Dims(cfg.R, ctx, cfg.d, cfg.n_heads, cfg.head_dim, cfg.ffn, cfg.V, 1, cfg.eps, cfg.rope_base,
                            binding.MTP_BF16)

    def size(ctx, prefix):
        return lib.mtp_draft_round_ext_workspace_bytes(ctypes.byref(dims(ctx)), 1, prefix)

    def call(ctx, prefix, ws_bytes):
        ext = binding.DraftExt()
        ext.prefix_k = ext.prefix_v = 1 << 20
        ext.prefix_len = prefix
        return lib.mtp_draft_round_ext(ctypes.byref(dims(ctx)), ctypes.byref(w), ctypes.byref(ext), *[fake] * 6, 1, 0, 0, fake,
                                       fake, None, fake, ws_bytes, None)

    most = 0x7FFFFF00  # rows of prefix and own cache together, as in mtp_prefix_attention
    assert size(300, most - 300) > 0 and call(300, most - 300, 16) == 4
    for ctx, prefix in ((300, most - 299), (300, 0x7FFFFFFF), (1 << 30, 1 << 30), (1, most)):
        assert size(ctx, prefix) == 0
        assert call(ctx, prefix, 1 << 60) == 2
