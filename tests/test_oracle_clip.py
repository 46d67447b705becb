"""Pins of the clipping and AdamW oracle (oracle/clip_adamw.py) against facts fixed outside
it.  CPU only."""

import math

import numpy as np
import pytest

from oracle import clip_adamw as O


def test_norms_by_hand():
    assert O.norm(np.array([3.0, -4.0]), "l2") == 5.0
    assert O.norm(np.array([3.0, -4.0]), "max") == 4.0
    # 2^2 + 3^2 + 6^2 = 49 over two tensors
    assert O.norm_of_tensors([np.array([[2.0], [-3.0]]), np.array([6.0])], "l2") == 7.0
    assert O.norm_of_tensors([np.array([2.0, -9.0]), np.array([6.0])], "max") == 9.0


@pytest.mark.parametrize("kind", ["l2", "max"])
def test_norm_of_non_finite_entries(kind):
    assert O.norm(np.array([1.0, -math.inf]), kind) == math.inf
    assert math.isnan(O.norm(np.array([1.0, math.nan, math.inf]), kind))


@pytest.mark.parametrize("kind", ["l2", "max"])
def test_norm_scales_and_ignores_order(kind):
    a = np.random.default_rng(11).standard_normal(1000)
    assert O.norm(-4.0 * a, kind) == pytest.approx(4.0 * O.norm(a, kind), rel=1e-14)
    assert O.norm(a[::-1].reshape(10, 100), kind) == pytest.approx(O.norm(a, kind), rel=1e-14)


def test_coefficient():
    assert O.coefficient(0.0, 1.0) == 1.0
    assert O.coefficient(1.0, 1.0) == 1.0
    assert O.coefficient(4.0, 1.0) == 0.25
    assert O.coefficient(math.inf, 1.0) == 0.0
    assert O.coefficient(math.inf, math.inf) == 1.0
    assert math.isnan(O.coefficient(math.nan, 1.0))


def test_first_adamw_step_by_hand():
    # t = 1 from zero moments: m_hat = g, v_hat = g^2, so x moves by lr * g / (|g| + eps)
    r = O.adamw([2.0, -2.0], [0.0, 0.0], [0.0, 0.0], [0.5, -0.25], 1, lr=0.1, beta1=0.9, beta2=0.99, eps=0.25,
                weight_decay=0.5)
    assert r.m == pytest.approx([0.05, -0.025])
    assert r.v == pytest.approx([0.0025, 0.000625])
    assert r.params == pytest.approx([2.0 - 0.1 - 0.1 * 0.5 / 0.75, -2.0 + 0.1 + 0.1 * 0.25 / 0.5])


def test_constant_gradient_keeps_its_corrected_moments():
    # with a constant gradient the corrected moments are g and g^2 at every step
    x, m, v = np.array([1.0]), np.zeros(1), np.zeros(1)
    for t in range(1, 40):
        r = O.adamw(x, m, v, [-3.0], t, lr=0.01, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
        assert r.params - x == pytest.approx(0.01 * 3.0 / (3.0 + 1e-8), rel=1e-9)
        x, m, v = r.params, r.m, r.v


def test_decay_is_decoupled():
    r = O.adamw([10.0], [0.0], [0.0], [0.0], 5, lr=0.1, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.2)
    assert r.params == pytest.approx([10.0 * (1 - 0.02)])
    assert r.m == 0 and r.v == 0
