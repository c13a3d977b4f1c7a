"""Refusals of the block norms' entry points, on the CPU: every call here fails
validation before any GPU call (fake pointers)."""
import math

import pytest

from int4_output_head_amd import binding
from tests.test_abi import declared_functions

EINVAL, EALIGN, EUNSUPPORTED = -1, -2, -5
A = 0x10000


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def test_header_declares_them():
    assert {"rms_norm_block_rows", "rms_norm_block_rows_int8"} <= set(declared_functions())


def block(lib, x=A, xs=64, r=A, rs=64, g=A, gs=64, act=0, dt=0, post=A, pre=A, wdt=0, scale=1.0, M=4, H=64, eps=1e-6,
          s=A, out=A, odt=0):
    return lib.rms_norm_block_rows(x, xs, r, rs, g, gs, act, dt, post, pre, wdt, scale, M, H, eps, s, out, odt, None)


def block8(lib, x=A, xs=64, r=A, rs=64, g=A, gs=64, act=0, dt=0, post=A, pre=A, wdt=0, c=A, scale=1.0, M=4, H=64,
           eps=1e-6, s=A, q=A, sc=A):
    return lib.rms_norm_block_rows_int8(x, xs, r, rs, g, gs, act, dt, post, pre, wdt, c, scale, M, H, eps, s, q, sc,
                                        None)


BOTH = [
    (dict(M=0), EINVAL), (dict(H=0), EINVAL), (dict(dt=3), EINVAL), (dict(wdt=-1), EINVAL), (dict(x=0), EINVAL),
    (dict(r=0), EINVAL), (dict(s=0), EINVAL), (dict(xs=63), EINVAL), (dict(rs=10), EINVAL), (dict(gs=63), EINVAL),
    (dict(gs=-64), EINVAL), (dict(g=0), EINVAL), (dict(act=2), EINVAL), (dict(act=-1), EINVAL),
    (dict(scale=math.inf), EINVAL), (dict(scale=math.nan), EINVAL), (dict(eps=-1e-6), EINVAL),
    (dict(eps=math.nan), EINVAL), (dict(x=A + 1), EALIGN), (dict(r=A + 1), EALIGN), (dict(g=A + 1), EALIGN),
    (dict(post=A + 1), EALIGN), (dict(pre=A + 1), EALIGN), (dict(s=A + 1), EALIGN), (dict(wdt=2, post=A + 2), EALIGN),
    (dict(H=8193, xs=9000, rs=9000, gs=9000), EUNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BOTH)
def test_refusals(lib, kw, status):
    assert block(lib, **kw) == status
    assert block8(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(odt=3), EINVAL), (dict(out=0), EINVAL), (dict(pre=0), EINVAL),
                                       (dict(out=A + 1), EALIGN)])
def test_refusals_of_the_norm(lib, kw, status):
    assert block(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [(dict(pre=0), EINVAL), (dict(q=0), EINVAL), (dict(sc=0), EINVAL),
                                       (dict(c=A + 1), EALIGN), (dict(sc=A + 2), EALIGN)])
def test_refusals_in_8_bits(lib, kw, status):
    assert block8(lib, **kw) == status
