"""YaRN's frequencies where the pair that turns once within the original length lies behind the last one, from the method's
definition ("YaRN: Efficient Context Window Extension of Large Language Models", 3.2 and its NTK-by-parts ramp over the pairs' index):
the ramp ends at the index, rounded up, of the pair that would turn beta_slow times, at rot - 1 at the most, whether there is such a
pair or not.  No GPU."""
import math

import numpy as np
import pytest

from deepseek_sequential_mtp_gb300 import build, lib as binding
from oracle import paged


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def published(rot, base, factor, original, slow, fast):
    dim = lambda turns: rot * np.log(original / (turns * 2 * np.pi)) / (2 * np.log(base))  # noqa: E731
    low, high = max(np.floor(dim(fast)), 0), min(np.ceil(dim(slow)), rot - 1)
    high = max(high, low + 0.001)  # (all pairs before the ramp, or a ramp of no width)
    ramp = np.clip((np.arange(rot // 2) - low) / (high - low), 0, 1)
    plain = base ** (-np.arange(0, rot, 2) / rot)
    return plain / factor * ramp + plain * (1 - ramp)


@pytest.mark.parametrize("rot,factor,original", [(64, 8.0, 131072.0), (128, 4.0, 65536.0), (24, 8.0, 32768.0), (64, 40.0, 4096.0),
                                                 (128, 8.0, 8192.0), (32, 16.0, 1048576.0), (64, 4.0, 1e12), (2, 4.0, 4096.0)])
@pytest.mark.parametrize("slow,fast", [(1.0, 32.0), (0.5, 8.0)])
def test_yarn(rot, factor, original, slow, fast):
    want = published(rot, 10000.0, factor, original, slow, fast)
    got, m = binding.rope_frequencies(rot, 10000.0, "yarn", factor, original, slow, fast, device="cpu")
    np.testing.assert_allclose(got.numpy(), want, rtol=1e-13)
    assert abs(m - (0.1 * math.log(factor) + 1)) < 1e-6
    np.testing.assert_allclose(paged.frequencies(rot, 10000.0, "yarn", factor, original, slow, fast)[0], want, rtol=1e-13)


def test_a_pair_between_the_two_ends():
    """The last of 32 pairs turns 2.78 times within 131072 positions: it lies within the ramp, which goes from pair 22 to 35."""
    f = binding.rope_frequencies(64, 10000.0, "yarn", 8.0, 131072.0, device="cpu")[0][-1].item()
    plain = 10000.0 ** (-62 / 64)
    assert 2.7 < 131072 * plain / (2 * math.pi) < 2.8
    share = (31 - 22) / (35 - 22)
    assert abs(f - plain * (share / 8 + 1 - share)) < 1e-12 * plain
