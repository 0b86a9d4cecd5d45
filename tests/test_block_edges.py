"""Calls of layer norm, the linear layer and AdamW at the edges of what they take, as
far as the C ABI decides them before any HIP call (the fake addresses are never
dereferenced)."""

import pytest

from momentum_compression_amd import onebit as ob
from tests.test_block_refusals import P, _linear_args


@pytest.fixture(scope="module")
def lib():
    return ob.load()


def test_round_dz_is_a_truth_value(lib):
    for bad in (-1, 2):
        assert lib.linear_backward(_linear_args(round_dz=bad), 9 * P, 1 << 30,
                                   None) == ob.ONEBIT_E_ARG
    # the workspace, which is checked last, stops these calls
    for good in (0, 1):
        assert lib.linear_backward(_linear_args(round_dz=good), None, 0,
                                   None) == ob.ONEBIT_E_WORKSPACE
