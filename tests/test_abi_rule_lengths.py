"""Histories and biases too long for a token's 31-bit count and entry number
are refused on the host (CPU; fake pointers, nothing is launched)."""
import pytest

from tests.test_abi_operators import A, EINVAL, EUNSUPPORTED, apply, lib, ruled, rules, verify  # noqa: F401


@pytest.mark.parametrize("call", [apply, verify, ruled])
@pytest.mark.parametrize("kw", [dict(n_history=2 ** 31 - 16), dict(n_history=2 ** 40), dict(n_bias=2 ** 31),
                                dict(n_bias=2 ** 62)])
def test_too_long(lib, call, kw):  # noqa: F811
    assert call(lib, r=rules(**kw)) == EUNSUPPORTED


@pytest.mark.parametrize("call", [apply, verify, ruled])
def test_other_errors_come_first(lib, call):  # noqa: F811
    assert call(lib, r=rules(n_history=2 ** 31, history_offsets=0)) == EINVAL
