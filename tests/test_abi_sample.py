"""Refusals of the sampler's entry point, on the CPU: every call here fails
validation before any GPU call (fake pointers)."""
import math

import pytest

from int4_output_head_amd import binding
from tests.test_abi import declared_functions

EINVAL, EALIGN, EWORKSPACE, EUNSUPPORTED = -1, -2, -3, -5
A = 0x10000


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def test_header_declares_them():
    assert {"sample_logits_rows", "sample_logits_workspace_bytes"} <= set(declared_functions())


def sample(lib, x=A, xs=100, dt=2, d=A, R=2, T=3, V=100, rules=None, s=(0, 0, 0, 0, 1.0, 0, 1.0, 0.0), u=A, acc=A,
           ids=A, probs=A, pd=A, na=A, ws=A, nb=1 << 40):
    s = None if s is None else binding._SAMPLING.pack(*s)
    return lib.sample_logits_rows(x, xs, dt, d, R, T, V, rules, s, u, acc, ids, probs, pd, na, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), EINVAL), (dict(dt=3), EINVAL), (dict(d=0), EINVAL), (dict(R=0), EINVAL), (dict(T=17), EINVAL),
    (dict(T=0), EINVAL), (dict(V=0), EINVAL), (dict(R=2000), EINVAL), (dict(xs=99), EINVAL), (dict(s=None), EINVAL),
    (dict(u=0), EINVAL), (dict(ids=0), EINVAL), (dict(probs=0), EINVAL), (dict(pd=0), EINVAL), (dict(na=0), EINVAL),
    (dict(ws=0), EINVAL), (dict(T=1, d=0), EINVAL),
    (dict(s=(0, 0, 0, 0, -0.1, 0, 1.0, 0.0)), EINVAL), (dict(s=(0, 0, 0, 0, math.inf, 0, 1.0, 0.0)), EINVAL),
    (dict(s=(0, 0, 0, 0, math.nan, 0, 1.0, 0.0)), EINVAL), (dict(s=(0, 0, 0, 0, 1.0, -1, 1.0, 0.0)), EINVAL),
    (dict(s=(0, 0, 0, 0, 1.0, 0, 1.1, 0.0)), EINVAL), (dict(s=(0, 0, 0, 0, 1.0, 0, math.nan, 0.0)), EINVAL),
    (dict(s=(0, 0, 0, 0, 1.0, 0, 1.0, -0.5)), EINVAL), (dict(s=(0, 0, 0, 0, 1.0, 0, 1.0, 2.0)), EINVAL),
    (dict(s=(A + 1, 0, 0, 0, 1.0, 0, 1.0, 0.0)), EALIGN), (dict(s=(0, A + 2, 0, 0, 1.0, 0, 1.0, 0.0)), EALIGN),
    (dict(s=(0, 0, A + 1, 0, 1.0, 0, 1.0, 0.0)), EALIGN), (dict(s=(0, 0, 0, A + 1, 1.0, 0, 1.0, 0.0)), EALIGN),
    (dict(x=A + 2), EALIGN), (dict(u=A + 1), EALIGN), (dict(acc=A + 1), EALIGN), (dict(ids=A + 2), EALIGN),
    (dict(probs=A + 1), EALIGN), (dict(pd=A + 1), EALIGN), (dict(na=A + 1), EALIGN), (dict(ws=A + 128), EALIGN),
    (dict(V=(1 << 24) + 1, xs=1 << 25), EUNSUPPORTED), (dict(nb=100), EWORKSPACE),
])
def test_refusals(lib, kw, status):
    assert sample(lib, **kw) == status


def test_workspace(lib):
    need = lib.sample_logits_workspace_bytes(2, 3, 100)
    assert need % 256 == 0 and need > 6 * 100 * 8
    assert sample(lib, nb=need - 1) == EWORKSPACE
    for sizes in ((0, 1, 10), (1, 17, 10), (1, 1, 0), (5000, 1, 10), (1, 1, (1 << 24) + 1)):
        assert lib.sample_logits_workspace_bytes(*sizes) == 0
