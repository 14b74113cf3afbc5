"""What a draft step over pages keeps of the cache that it was built with (no GPU: nothing is launched)."""
import gc
import weakref
from dataclasses import replace

import pytest
import torch

from deepseek_sequential_mtp_gb300 import build, lib, synth


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def cache(cfg, page, eight):
    n = cfg.R * cfg.ctx // page
    c = {"page_table": torch.arange(n, dtype=torch.int32).view(cfg.R, -1)}
    for name in ("k", "v"):
        c[name + "_pages"] = torch.zeros((n, cfg.n_heads, page, cfg.head_dim), dtype=torch.uint8 if eight else torch.bfloat16)
        if eight:
            c[name + "_scale"] = torch.zeros((n, cfg.n_heads, page // 16), dtype=torch.uint8)
    return c


@pytest.mark.parametrize("eight", [True, False])
@pytest.mark.parametrize("gamma", [0, 3])
def test_the_tensors_live_as_long_as_the_step(eight, gamma):
    """The step reads the addresses that it was given: a dict whose entries are replaced or taken out does not free them."""
    cfg = replace(synth.DRAFT_SMALL, ctx=320)
    w = synth.make_draft_inputs(cfg, 1)["weights"]
    c = cache(cfg, 32, eight)
    seen = {k: weakref.ref(t) for k, t in c.items()}
    at = {k: t.data_ptr() for k, t in c.items()}
    step = lib.DraftRound(cfg, w, gamma, device="cpu", paged=c) if gamma else lib.DraftStep(cfg, w, device="cpu", paged=c)
    c["page_table"] = c["page_table"] + 1
    for k in list(c):
        if k != "page_table":
            del c[k]
    del c
    gc.collect()
    for k, t in seen.items():
        assert t() is not None and t().data_ptr() == at[k], k
    s = step.paged
    names = {"k": "k_pages", "v": "v_pages", "page_table": "page_table", **({"k_scale": "k_scale", "v_scale": "v_scale"} if eight else {})}
    assert {k: getattr(s, f) for f, k in names.items()} == at
    del step
    gc.collect()
    assert all(t() is None for t in seen.values())


@pytest.mark.parametrize("name", ["k_pages", "v_pages", "page_table"])
@pytest.mark.parametrize("how", ["missing", "none"])
def test_a_cache_without_its_tensors_is_refused(name, how):
    cfg = replace(synth.DRAFT_SMALL, ctx=320)
    w = synth.make_draft_inputs(cfg, 1)["weights"]
    c = cache(cfg, 32, False)
    if how == "none":
        c[name] = None
    else:
        del c[name]
    with pytest.raises(lib.MtpError, match=name):
        lib.DraftStep(cfg, w, device="cpu", paged=c)
