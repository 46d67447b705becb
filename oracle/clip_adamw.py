"""Plain CPU oracle of the gradient norms, clipping and the AdamW step (include/psgd_clip.h).

TEST INFRASTRUCTURE.  Only the test suite and the package smoke check may import this
module.  The GPU library never calls it and shares no code with it.

Everything is float64 on the values of the inputs, from the definitions:

* norm: square root of the sum of squares, or the largest magnitude; a NaN entry makes
  either NaN;
* clipping coefficient: 1 where the norm is at most the bound, else bound / norm (0 for an
  infinite norm, NaN for a NaN norm);
* AdamW (decoupled weight decay, bias-corrected moments) on the scaled gradient.

Pinned by tests/test_oracle_clip.py: values computed by hand, scaling and permutation
properties, and the closed form of a constant gradient.
"""

from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Sequence

import numpy as np


def norm(values: np.ndarray, kind: str) -> float:
    """Norm of all the entries of `values` ("l2" or "max")."""
    a = np.abs(np.asarray(values, dtype=np.float64)).ravel()
    if np.isnan(a).any():
        return math.nan
    if np.isinf(a).any():
        return math.inf
    return float(a.max()) if kind == "max" else float(np.sqrt(np.sum(a * a)))


def norm_of_tensors(tensors: Sequence[np.ndarray], kind: str) -> float:
    """Norm over many tensors: of the concatenation of their entries."""
    return norm(np.concatenate([np.asarray(t, dtype=np.float64).ravel() for t in tensors]), kind)


def coefficient(n: float, max_norm: float) -> float:
    if n <= max_norm:
        return 1.0
    return math.nan if math.isnan(n) else max_norm / n


@dataclass
class AdamwResult:
    params: np.ndarray
    m: np.ndarray
    v: np.ndarray


def adamw(x, m, v, g, t: int, lr: float, beta1: float, beta2: float, eps: float, weight_decay: float) -> AdamwResult:
    """Step number t (the first is 1) on gradient g (already scaled)."""
    x, m, v, g = (np.asarray(a, dtype=np.float64) for a in (x, m, v, g))
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    m_hat = m / (1.0 - beta1 ** t)
    v_hat = v / (1.0 - beta2 ** t)
    x = x - lr * weight_decay * x - lr * m_hat / (np.sqrt(v_hat) + eps)
    return AdamwResult(x, m, v)
