"""Host-side checks of the limits of the scaled cache's writes (no GPU is needed)."""
import ctypes

import pytest

from kv_cache_injection_gb300 import _lib, build
from tests.test_scaled_refusals import CODES, SCALES, move_args
from tests.test_serve_refusals import INVALID, append_args


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def append_within(lib, args, budget):
    return lib.is_append_scaled_within(ctypes.byref(args), SCALES, budget, None)


def move_within(lib, args, budget):
    return lib.is_move_scaled_within(ctypes.byref(args), budget, None)


@pytest.mark.parametrize("budget", [-1, 2_000_000_001, -(1 << 63), (1 << 63) - 1])
def test_writes_refuse_budgets(lib, budget):
    for within, args in ((append_within, append_args(num_tokens=0, cache=CODES)), (move_within, move_args(num_tokens=0))):
        assert within(lib, args, budget) == INVALID
        assert b"budget_ns" in lib.is_last_error_message()


def test_writes_take_their_range(lib):
    for budget in (0, 1, 2_000_000_000):
        assert append_within(lib, append_args(num_tokens=0, cache=CODES), budget) == 0
        assert move_within(lib, move_args(num_tokens=0), budget) == 0
    assert lib.is_append_scaled_within(None, SCALES, 0, None) == INVALID and lib.is_move_scaled_within(None, 0, None) == INVALID


def test_writes_with_a_limit_refuse_what_the_others_refuse(lib):
    assert append_within(lib, append_args(cache=CODES, k=None), 5) == INVALID
    assert move_within(lib, move_args(scales=None), 5) == INVALID
