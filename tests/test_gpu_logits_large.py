"""mtp_logits_probs at the corners of its sizes: the largest vocabularies together with the
largest histories, whose tables of marked ids fill a CTA's shared memory.

Tolerance: the bar of test_gpu_logits.py."""
import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib

from test_gpu_logits import _check, _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,H,used", [
    (400000, 32768, 32768), (524288, 30000, 30000), (524288, 262144, 262144),
    (524288, 262144, 5),        # a short text in a large buffer
    (524287, 262144, 262143),   # rows that are not 16-byte aligned
])
def test_long_histories_beside_large_vocabularies(V, H, used):
    a = _inputs(2, 2, V, torch.float32, 1, 3, True, V % 1000 + H)
    ids = np.random.default_rng(H).permutation(V)[:H].astype(np.int32)  # distinct: every one has a place of its own
    a["hist"] = torch.from_numpy(np.stack([ids, np.roll(ids, 7)]))
    # half of the second request's ids within one slice of 32768, each some 8 times
    a["hist"][1, : H // 2] %= 16384
    a["hist_len"] = torch.tensor([used, max(1, used - 3)], dtype=torch.int32)
    a["prompt_len"] = torch.tensor([used // 3, 0], dtype=torch.int32)
    _check(a, _run(a))


def test_a_history_of_one_slice():
    """Every entry of a slice of 32768 marked, and all counts on a few ids."""
    V = 524288
    a = _inputs(1, 1, V, torch.bfloat16, 1, 3, False, 7)
    a["hist"] = torch.arange(262144, dtype=torch.int32)[None] % 32768 + 5 * 32768
    a["hist_len"] = torch.tensor([262144], dtype=torch.int32)
    a["prompt_len"] = torch.tensor([100], dtype=torch.int32)
    a["frequency"] = torch.tensor([0.25])
    _check(a, _run(a))


def test_most_of_everything():
    """The largest list of marked ids that the limits allow: history, drafts and biases."""
    V, L = 524288, 40
    a = _inputs(1, L, V, torch.bfloat16, 1, 4095, True, 8)
    a["hist"] = (torch.arange(262144, dtype=torch.int32) * 2)[None]
    a["hist_len"] = torch.tensor([262144], dtype=torch.int32)
    a["prompt_len"] = torch.tensor([200000], dtype=torch.int32)
    p, st = _run(a)
    assert (st == 0).all()
    last = {k: (v[:, L - 1:] if k in ("logits", "mask") else v) for k, v in a.items()}
    last["hist"] = torch.cat([a["hist"], a["draft"]], 1)  # the last row's text: history and all drafts
    last["hist_len"] = torch.tensor([262144 + L - 1], dtype=torch.int32)
    last["draft"] = None
    _check(last, (p[:, L - 1:], st[:, L - 1:]))
