"""Refusals of the 4-bit floating-point entry points, on the CPU: every call
here fails validation before any GPU call (fake pointers)."""
import pytest

from int4_output_head_amd import binding
from tests.test_abi import declared_functions

EINVAL, EALIGN, EWORKSPACE, EUNSUPPORTED = -1, -2, -3, -5
A = 0x10000


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def test_header_declares_them():
    assert {"quantize_rows_mxfp4", "dequantize_rows_mxfp4", "linear_mxfp4_rows",
            "linear_mxfp4_rows_workspace_bytes"} <= set(declared_functions())


def quantize(lib, x=A, xs=64, dt=0, M=4, H=64, q=A, s=A):
    return lib.quantize_rows_mxfp4(x, xs, dt, M, H, q, s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), EINVAL), (dict(q=0), EINVAL), (dict(s=0), EINVAL), (dict(M=0), EINVAL), (dict(H=0), EINVAL),
    (dict(H=16), EINVAL), (dict(H=48), EINVAL), (dict(dt=3), EINVAL), (dict(xs=63), EINVAL), (dict(xs=-64), EINVAL),
    (dict(x=A + 1), EALIGN), (dict(dt=2, x=A + 2), EALIGN), (dict(q=A + 2), EALIGN),
    (dict(H=65568, xs=65568), EUNSUPPORTED), (dict(H=65536, xs=65536, M=1 << 24), EUNSUPPORTED),
])
def test_quantize_refusals(lib, kw, status):
    assert quantize(lib, **kw) == status


def dequantize(lib, q=A, s=A, M=4, H=64, out=A, dt=0):
    return lib.dequantize_rows_mxfp4(q, s, M, H, out, dt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), EINVAL), (dict(s=0), EINVAL), (dict(out=0), EINVAL), (dict(M=0), EINVAL), (dict(H=33), EINVAL),
    (dict(dt=-1), EINVAL), (dict(q=A + 8), EALIGN), (dict(out=A + 1), EALIGN), (dict(H=65568), EUNSUPPORTED),
    (dict(H=65536, M=1 << 24), EUNSUPPORTED),
])
def test_dequantize_refusals(lib, kw, status):
    assert dequantize(lib, **kw) == status


def linear(lib, c=A, s=A, w=A, ws=A, b=A, act=0, r=A, rs=8, M=4, N=8, K=64, out=A, ldo=8, dt=0, work=A, nb=1 << 30):
    return lib.linear_mxfp4_rows(c, s, w, ws, b, act, r, rs, M, N, K, out, ldo, dt, work, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), EINVAL), (dict(N=0), EINVAL), (dict(K=16), EINVAL), (dict(K=48), EINVAL), (dict(c=0), EINVAL),
    (dict(s=0), EINVAL), (dict(w=0), EINVAL), (dict(ws=0), EINVAL), (dict(out=0), EINVAL), (dict(act=4), EINVAL),
    (dict(act=-1), EINVAL), (dict(dt=3), EINVAL), (dict(ldo=7), EINVAL), (dict(rs=7), EINVAL),
    (dict(c=A + 8), EALIGN), (dict(w=A + 4), EALIGN), (dict(b=A + 1), EALIGN), (dict(r=A + 1), EALIGN),
    (dict(out=A + 1), EALIGN), (dict(K=65568), EUNSUPPORTED),
    (dict(N=(1 << 24) + 1, ldo=1 << 25, rs=1 << 25), EUNSUPPORTED), (dict(M=(1 << 20) + 1), EUNSUPPORTED),
    (dict(M=1 << 20, N=1 << 20, ldo=1 << 20, rs=1 << 20), EUNSUPPORTED),
])
def test_linear_refusals(lib, kw, status):
    assert linear(lib, **kw) == status


def test_linear_workspace(lib):
    need = lib.linear_mxfp4_rows_workspace_bytes(4, 64, 16384)       # the stream splits K above 8192
    assert need >= 2 * 4 * 64 * 4 and need % 256 == 0
    big = dict(M=4, N=64, K=16384, ldo=64, rs=64)
    assert linear(lib, work=0, **big) == EINVAL
    assert linear(lib, work=A + 128, **big) == EALIGN
    assert linear(lib, nb=need - 1, **big) == EWORKSPACE
    assert lib.linear_mxfp4_rows_workspace_bytes(4, 64, 64) == 0
    assert lib.linear_mxfp4_rows_workspace_bytes(0, 64, 64) == 0
    assert lib.linear_mxfp4_rows_workspace_bytes(4, 64, 65568) == 0
