"""Host-side checks of the serving step's calls beside their struct fields (no GPU is needed)."""
import ctypes

import pytest

from kv_cache_injection_gb300 import _lib, api, build
from tests.test_serve_refusals import INVALID, attend_args


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("budget", [-1, 2_000_000_001, -(1 << 63), (1 << 63) - 1])
def test_attend_within_refuses_budgets(lib, budget):
    args = attend_args(num_tokens=0)
    assert lib.is_attend_within(ctypes.byref(args), budget, None) == INVALID
    assert b"budget_ns" in lib.is_last_error_message()


def test_attend_within_takes_its_range(lib):
    args = attend_args(num_tokens=0)
    assert [lib.is_attend_within(ctypes.byref(args), b, None) for b in (0, 1, 2_000_000_000)] == [0, 0, 0]
    assert lib.is_attend_within(None, 0, None) == INVALID


def test_extend_says_that_it_needs_a_status_word():
    with pytest.raises(ValueError, match="status_out is required"):
        api.is_extend_block_table(None, None, None, 16, 4, None, None)
