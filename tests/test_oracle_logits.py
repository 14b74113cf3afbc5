"""The logits oracle: closed forms and worked rows."""
import math

import numpy as np
import pytest

from oracle import logits as ol


def test_plain_softmax_and_temperature():
    x = np.log(np.array([1.0, 2.0, 5.0]))
    p, st = ol.row(x, [], [])
    assert st == ol.OK
    np.testing.assert_allclose(p, [0.125, 0.25, 0.625], rtol=1e-14)
    p, _ = ol.row(x, [], [], temperature=0.5)  # squares the odds
    np.testing.assert_allclose(p, np.array([1, 4, 25]) / 30, rtol=1e-14)
    p, _ = ol.row([1.0, 3.0, 3.0], [], [], temperature=0.0)
    assert p.tolist() == [0, 1, 0]


def test_penalties_worked():
    """Token 0 in the prompt only, 1 generated twice, 2 once, 3 never; the
    repetition penalty divides a positive logit and multiplies a negative one."""
    x = [2.0, 4.0, -1.0, 0.5]
    p, st = ol.row(x, [0], [1, 2, 1], repetition=2.0, frequency=0.25, presence=0.5)
    z = np.array([1.0, 2.0 - 0.5 - 0.5, -2.0 - 0.25 - 0.5, 0.5])
    np.testing.assert_allclose(p, np.exp(z) / np.exp(z).sum(), rtol=1e-14)
    assert st == ol.OK


def test_bias_and_mask():
    p, _ = ol.row([0.0, 0.0, 0.0], [], [], biases=[(1, 9.0), (1, math.log(2.0)), (-1, 5.0), (3, 5.0)])
    np.testing.assert_allclose(p, [0.25, 0.5, 0.25], rtol=1e-14)
    p, _ = ol.row([0.0, 7.0, math.log(3.0)], [], [], allowed=[True, False, True])
    np.testing.assert_allclose(p, [0.25, 0.0, 0.75], rtol=1e-14)
    assert ol.unpack_mask(np.array([-2147483647], dtype=np.int32), 32).nonzero()[0].tolist() == [0, 31]


@pytest.mark.parametrize("kw,status", [
    (dict(x=[-np.inf, -np.inf]), ol.EMPTY),
    (dict(x=[0.0, 1.0], allowed=[False, False]), ol.EMPTY),
    (dict(x=[0.0, np.nan]), ol.INVALID),
    (dict(x=[0.0, np.inf]), ol.INVALID),
    (dict(x=[0.0, np.nan], allowed=[True, False]), ol.OK),
    (dict(x=[0.0, 1.0], temperature=-1.0), ol.INVALID_PARAM),
    (dict(x=[0.0, 1.0], repetition=0.0), ol.INVALID_PARAM),
    (dict(x=[0.0, 1.0], presence=np.nan), ol.INVALID_PARAM)])
def test_status(kw, status):
    p, st = ol.row(kw.pop("x"), [], [], **kw)
    assert st == status
    assert (p.sum() == pytest.approx(1.0)) if st == ol.OK else (p == 0).all()
