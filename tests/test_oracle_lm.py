"""Pins of the oracle of dropout, embedding and cross entropy: published words of the
generator, closed forms, and gradients against differences.  CPU only."""

import numpy as np
import pytest

from oracle import lm as O


def test_generator_gives_the_published_words():
    """Known answers that the generator's authors publish with it (Random123, philox4x32, 10 rounds)."""
    pi = [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344]
    for counter, key, words in [
        ([0] * 4, (0, 0), [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
        ([0xFFFFFFFF] * 4, (0xFFFFFFFF, 0xFFFFFFFF), [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
        (pi, (0xA4093822, 0x299F31D0), [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
    ]:
        assert O.philox4x32([counter], key)[0].tolist() == words


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.93, 1.0])
def test_share_of_kept_entries(p):
    n = 200000
    keep = O.kept((n,), p, 77, 5)
    # five standard deviations of a binomial share
    assert abs(keep.mean() - (1 - p)) <= 5 * np.sqrt(p * (1 - p) / n)
    x = np.ones(n)
    values = [1.0] if p == 0 else [0.0] if p == 1 else [0.0, 1 / (1 - p)]
    assert np.array_equal(np.unique(O.dropout(x, (p, 77, 5))), values)


def test_masks_differ_by_seed_step_and_place():
    base = O.kept((4096,), 0.5, 7, 1)
    for other in (O.kept((4096,), 0.5, 8, 1), O.kept((4096,), 0.5, 7, 2), O.kept((4096,), 0.5, 7 + (1 << 32), 1),
                  O.kept((4096,), 0.5, 7, 1 + (1 << 32)), np.roll(base, 1), np.roll(base, 4)):
        assert 0.4 < (other == base).mean() < 0.6


def _case(seed=0, W=2, T=5, V=11, d=4):
    rng = np.random.default_rng(seed)
    x, table = rng.standard_normal((W, T, d)), rng.standard_normal((V, d))
    targets = rng.integers(0, V, (W, T))
    targets[0, 1], targets[1, 3] = -100, V
    return x, table, targets


def test_uniform_scores_give_log_vocab():
    x, table, targets = _case()
    losses, lse, mean = O.loss(0 * x, table, targets)
    ok = (targets >= 0) & (targets < len(table))
    assert np.allclose(losses, ok * np.log(len(table)), rtol=1e-14) and np.allclose(mean, np.log(len(table)), rtol=1e-14)
    assert np.array_equal(lse == 0, ~ok)


def test_one_word_is_certain():
    x, table, _ = _case(V=1)
    targets = np.zeros(x.shape[:2], dtype=np.int64)
    losses, lse, _ = O.loss(x, table, targets)
    assert np.all(np.abs(losses) < 1e-14)
    dx, g = O.loss_grad(x, table, targets, lse)
    assert np.all(np.abs(dx) < 1e-14) and np.all(np.abs(g) < 1e-14)


def test_gradients_sum_to_nothing_over_the_vocabulary():
    x, table, targets = _case()
    _, lse, _ = O.loss(x, table, targets)
    g, _ = O.score_grad(x, table, targets, lse)
    assert np.allclose(g.sum(-1), 0, atol=1e-15)


@pytest.mark.parametrize("drop", [None, (0.4, 3, 9)])
@pytest.mark.parametrize("scaled", [False, True])
def test_loss_gradient_against_differences(drop, scaled):
    x, table, targets = _case(3)
    scale = np.array([0.7, -3.0]) if scaled else None
    weight = np.ones(2) if scale is None else scale
    _, lse, _ = O.loss(x, table, targets, drop)
    dx, g = O.loss_grad(x, table, targets, lse, scale, drop)
    h = 1e-5
    for a, grad in ((x, dx), (table, g.sum(0))):
        num = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            old = a[i]
            vals = []
            for s in (h, -h):
                a[i] = old + s
                vals.append(O.loss(x, table, targets, drop)[2] @ weight)
            a[i] = old
            num[i] = (vals[0] - vals[1]) / (2 * h)
        # the differences' own error: h^2 times a third derivative of order 10, and rounding over h
        assert np.abs(num - grad).max() < 1e-8


@pytest.mark.parametrize("drop", [None, (0.4, 3, 9)])
def test_embedding_gradient_is_the_adjoint(drop):
    rng = np.random.default_rng(5)
    table, dy = rng.standard_normal((6, 3)), rng.standard_normal((2, 9, 3))
    tokens = rng.integers(-1, 7, (2, 9))
    g = O.embed_grad(6, tokens, dy, drop)
    assert np.isclose((O.embed(table, tokens, drop) * dy).sum(), (g.sum(0) * table).sum(), rtol=1e-12)
    assert np.all(O.embed(table, tokens)[(tokens < 0) | (tokens > 5)] == 0)
