"""Limits of the language-model part of the C ABI, without a GPU (no call here reaches a device)."""

import pytest

from distributed_sgd_gradient_ef_amd import psgd
from tests.test_abi_lm import INVALID, _dropout

pytestmark = pytest.mark.usefixtures("built_library")


@pytest.mark.parametrize("rows,cols", [(1 << 31, 1 << 10), (1, 1 << 41), (1 << 41, 1), ((1 << 41) // 3 + 1, 3)])
def test_dropout_refuses_from_two_to_the_41(rows, cols):
    x, out = 1 << 44, 1 << 45
    assert _dropout(x=x, xs=cols, out=out, os=cols, rows=rows, cols=cols) == INVALID
    assert b"2^41" in psgd.load_library().psgd_last_error()
