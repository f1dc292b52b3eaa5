"""Forks that would keep one workgroup walking a table for minutes are refused (CPU: before any HIP call, with fake
addresses): more forks than the table has rows, each of a very wide row, or more private entries than a pool has pages."""
import pytest

from test_cache_abi import _fork, _lib


@pytest.mark.parametrize("over", [
    dict(n=1024, R=1, W=1 << 26, priv=0), dict(n=1024, R=64, W=(1 << 16) + 1, priv=1), dict(n=2, R=1, W=1 << 26, priv=0),
    dict(n=1, R=2, W=1 << 25, priv=1 << 25), dict(n=1, R=4, W=65537, priv=65537), dict(n=0, R=4, W=65537, priv=65537),
])
def test_forks_without_end_are_refused(over):
    assert _fork(_lib(), **over) == 2


@pytest.mark.parametrize("over", [dict(n=1024, R=64, W=1 << 16, priv=1), dict(n=1, R=1, W=1 << 26, priv=0), dict(n=4, R=4, W=1 << 20, priv=65536)])
def test_forks_up_to_the_limits_pass_the_size_check(over):
    """(Seen from the next check on: a missing table.)"""
    assert _fork(_lib(), table=None, **over) == 1
