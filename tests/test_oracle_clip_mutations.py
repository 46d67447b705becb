"""Plant mistakes in (a patched copy of) the clipping and AdamW oracle and check that the
pins in test_oracle_clip.py catch every one of them.  CPU only; pytest's monkeypatch
restores the real module after each case."""

import math

import numpy as np
import pytest

from oracle import clip_adamw as O
from tests import test_oracle_clip as T


def _pins():
    for kind in ("l2", "max"):
        yield lambda kind=kind: T.test_norm_of_non_finite_entries(kind)
        yield lambda kind=kind: T.test_norm_scales_and_ignores_order(kind)
    yield from (T.test_norms_by_hand, T.test_coefficient, T.test_first_adamw_step_by_hand,
                T.test_constant_gradient_keeps_its_corrected_moments, T.test_decay_is_decoupled)


def _adamw(coupled=False, eps_inside=False, correct_m=True, correct_v=True, old_t=False, square=True):
    def adamw(x, m, v, g, t, lr, beta1, beta2, eps, weight_decay):
        x, m, v, g = (np.asarray(a, dtype=np.float64) for a in (x, m, v, g))
        t = max(t - 1, 1) if old_t else t
        g = g + weight_decay * x if coupled else g
        m = beta1 * m + (1.0 - beta1) * g
        v = beta2 * v + (1.0 - beta2) * (g * g if square else np.abs(g))
        m_hat = m / (1.0 - beta1 ** t) if correct_m else m
        v_hat = v / (1.0 - beta2 ** t) if correct_v else v
        den = np.sqrt(v_hat + eps) if eps_inside else np.sqrt(v_hat) + eps
        x = x - (0.0 if coupled else lr * weight_decay * x) - lr * m_hat / den
        return O.AdamwResult(x, m, v)
    return adamw


def _norm(f):
    return lambda values, kind: f(np.abs(np.asarray(values, dtype=np.float64)).ravel(), kind)


_REAL = O.norm
MUTATIONS = {
    "norm without the root": ("norm", _norm(lambda a, k: _REAL(a, k) ** (2 if k == "l2" else 1))),
    "sum of magnitudes": ("norm", _norm(lambda a, k: float(a.sum()) if k == "l2" else _REAL(a, k))),
    "largest entry, not magnitude": ("norm", lambda v, k: float(np.max(v)) if k == "max" else _REAL(v, k)),
    "NaN ignored": ("norm", _norm(lambda a, k: _REAL(np.nan_to_num(a, nan=0.0, posinf=math.inf), k))),
    "norm of the first tensor": ("norm_of_tensors", lambda ts, k: _REAL(ts[0], k)),
    "sum of the tensors' norms": ("norm_of_tensors", lambda ts, k: sum(_REAL(t, k) for t in ts)),
    "always scaled to the bound": ("coefficient", lambda n, c: c / n if n else 1.0),
    "scaled by the norm's inverse": ("coefficient", lambda n, c: 1.0 if n <= c else 1.0 / n ** 2),
    "NaN taken for small": ("coefficient", lambda n, c: 1.0 if not n > c else c / n),
    "coupled decay": ("adamw", _adamw(coupled=True)),
    "eps inside the root": ("adamw", _adamw(eps_inside=True)),
    "first moment not corrected": ("adamw", _adamw(correct_m=False)),
    "second moment not corrected": ("adamw", _adamw(correct_v=False)),
    "step count one behind": ("adamw", _adamw(old_t=True)),
    "magnitudes instead of squares": ("adamw", _adamw(square=False)),
}


def _caught():
    for pin in _pins():
        try:
            with np.errstate(all="ignore"):
                pin()
        except (AssertionError, ZeroDivisionError):
            return True
    return False


def test_no_mutation_passes():
    assert not _caught()


@pytest.mark.parametrize("name", MUTATIONS)
def test_mutation_is_caught(name, monkeypatch):
    where, what = MUTATIONS[name]
    monkeypatch.setattr(O, where, what)
    assert _caught(), name
