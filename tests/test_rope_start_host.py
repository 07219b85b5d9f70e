"""Where a rotation's positions may start (no GPU needed)."""
import pytest

from learned_kv_cache_gb300 import rope


@pytest.mark.parametrize("start", [0, 5, -7, 2 ** 31 - 1, -2 ** 31])
def test_a_start_that_fits(start):
    assert rope._start(start) == start


@pytest.mark.parametrize("start", [2 ** 31, -2 ** 31 - 1, 2 ** 32 + 7, 2 ** 64])
def test_a_start_that_does_not(start):
    with pytest.raises(ValueError):
        rope._start(start)
