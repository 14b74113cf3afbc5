"""The 4-bit weight oracle and the synthetic quantiser, by hand and by bounds."""
import numpy as np
import pytest
import torch

from deepseek_sequential_mtp_gb300 import synth
from oracle import int4 as oi


def test_dequantize_worked():
    q = np.array([[0x10, 0xF8], [0x7A, 0x03]], dtype=np.uint8)  # codes 0 1 8 15 / 10 7 3 0
    s = np.array([[0.5, 2.0], [1.0, -4.0]])
    z = np.array([[0, 8], [24, 3]], dtype=np.uint8)  # only the low four bits count: 24 is 8
    np.testing.assert_array_equal(oi.dequantize(q, s, z, 2), [[0.0, 0.5, 0.0, 14.0], [2.0, -1.0, 0.0, 12.0]])
    np.testing.assert_array_equal(oi.dequantize(q, s, None, 2), [[-4.0, -3.5, 0.0, 14.0], [2.0, -1.0, 20.0, 32.0]])
    np.testing.assert_array_equal(oi.dequantize(q, s[:, :1], None, 4)[0], [-4.0, -3.5, 0.0, 3.5])


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("n,K,group", [(5, 96, 64), (7, 128, 32), (3, 160, 128)])
def test_quantiser_is_within_half_a_step(n, K, group, symmetric):
    w = torch.randn(n, K, generator=torch.Generator().manual_seed(K)).to(torch.bfloat16)
    q, s, z = synth.quantize_int4_groups(w, group, symmetric)
    assert q.shape == (n, K // 2) and s.shape == (n, -(-K // group)) and (z is None) == symmetric
    W = oi.dequantize(q.numpy(), s.double().numpy(), None if z is None else z.numpy(), group)
    step = s.double().numpy()[:, np.arange(K) // group]
    # rounding to the nearest code: half a step, and the bf16 rounding of the scale moves the
    # outermost codes by 8 (16 with a zero point) times 2^-8 of a step besides
    slack = 0.5 + (8 if symmetric else 16) * 2.0 ** -8 + (1.0 if symmetric else 0.5)
    assert (np.abs(W - w.double().numpy()) <= slack * step).all()
