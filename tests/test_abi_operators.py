"""Refusals of the row, linear and logit-rule entry points, on the CPU: every
call here fails validation before any GPU call (fake pointers)."""
import ctypes
import math

import pytest
import torch

from int4_output_head_amd import binding
from tests.test_abi import declared_functions

OK, EINVAL, EALIGN, EWORKSPACE, EHIP, EUNSUPPORTED = 0, -1, -2, -3, -4, -5
A = 0x10000


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def test_headers_declare_the_operators():
    names = declared_functions()
    for n in ("rms_norm_rows", "rms_norm_rows_int8", "quantize_rows_int8", "linear_int4_rows",
              "linear_int4_rows_workspace_bytes", "logit_rules_apply", "logit_rules_verify",
              "logit_rules_verify_workspace_bytes", "verify_lm_head_int4_ruled",
              "verify_lm_head_int4_ruled_workspace_bytes"):
        assert n in names, n


def norm(lib, x=A, xs=64, r=A, rs=64, dt=0, w=A, wdt=0, M=4, H=64, eps=1e-6, s=A, out=A, odt=0):
    return lib.rms_norm_rows(x, xs, r, rs, dt, w, wdt, M, H, eps, s, out, odt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), EINVAL), (dict(H=0), EINVAL), (dict(dt=3), EINVAL), (dict(wdt=-1), EINVAL), (dict(odt=7), EINVAL),
    (dict(x=0), EINVAL), (dict(w=0), EINVAL), (dict(out=0), EINVAL), (dict(xs=63), EINVAL), (dict(rs=10), EINVAL),
    (dict(xs=-64), EINVAL), (dict(r=0), EINVAL), (dict(eps=-1e-6), EINVAL), (dict(eps=math.inf), EINVAL),
    (dict(eps=math.nan), EINVAL), (dict(x=A + 1), EALIGN), (dict(r=A + 1), EALIGN), (dict(w=A + 1), EALIGN),
    (dict(out=A + 1), EALIGN), (dict(s=A + 1), EALIGN), (dict(dt=2, x=A + 2), EALIGN),
    (dict(H=8193, xs=9000, rs=9000), EUNSUPPORTED),
])
def test_norm_refusals(lib, kw, status):
    assert norm(lib, **kw) == status


def norm8(lib, x=A, xs=64, r=A, rs=64, dt=0, w=A, wdt=0, c=A, M=4, H=64, eps=1e-6, s=A, q=A, sc=A):
    return lib.rms_norm_rows_int8(x, xs, r, rs, dt, w, wdt, c, M, H, eps, s, q, sc, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), EINVAL), (dict(w=0), EINVAL), (dict(q=0), EINVAL), (dict(sc=0), EINVAL), (dict(r=0), EINVAL),
    (dict(c=A + 1), EALIGN), (dict(sc=A + 2), EALIGN), (dict(H=8200, xs=8200, rs=8200), EUNSUPPORTED),
    (dict(eps=-0.5), EINVAL), (dict(xs=1), EINVAL),
])
def test_norm8_refusals(lib, kw, status):
    assert norm8(lib, **kw) == status


@pytest.mark.parametrize("args,status", [
    ((0, 64, 0, A, 4, 64, A, A), EINVAL), ((A, 64, 5, A, 4, 64, A, A), EINVAL), ((A, 60, 0, A, 4, 64, A, A), EINVAL),
    ((A, 64, 0, A, 4, 64, 0, A), EINVAL), ((A, 64, 0, A, 4, 64, A, 0), EINVAL), ((A, 64, 0, A + 1, 4, 64, A, A), EALIGN),
    ((A, 65537, 0, A, 4, 65537, A, A), EUNSUPPORTED),
])
def test_quantize_refusals(lib, args, status):
    assert lib.quantize_rows_int8(*args, None) == status


def linear(lib, c=A, cs=64, s=A, w=A, os=A, b=A, act=0, r=A, rs=8, M=4, N=8, K=64, out=A, ldo=8, dt=0, ws=A,
           nb=1 << 30):
    return lib.linear_int4_rows(c, cs, s, w, os, b, act, r, rs, M, N, K, out, ldo, dt, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=0), EINVAL), (dict(N=0), EINVAL), (dict(K=16), EINVAL), (dict(K=48), EINVAL), (dict(c=0), EINVAL),
    (dict(s=0), EINVAL), (dict(w=0), EINVAL), (dict(out=0), EINVAL), (dict(act=4), EINVAL), (dict(act=-1), EINVAL),
    (dict(dt=3), EINVAL), (dict(cs=32), EINVAL), (dict(ldo=7), EINVAL), (dict(rs=7), EINVAL),
    (dict(c=A + 8), EALIGN), (dict(cs=72), EALIGN), (dict(w=A + 4), EALIGN), (dict(s=A + 2), EALIGN),
    (dict(os=A + 1), EALIGN), (dict(b=A + 1), EALIGN), (dict(r=A + 1), EALIGN), (dict(out=A + 1), EALIGN),
    (dict(K=65568, cs=65568), EUNSUPPORTED), (dict(N=(1 << 24) + 1, ldo=1 << 25, rs=1 << 25), EUNSUPPORTED),
    (dict(M=(1 << 20) + 1), EUNSUPPORTED),
    (dict(M=1 << 20, N=1 << 20, ldo=1 << 20, rs=1 << 20), EUNSUPPORTED),
])
def test_linear_refusals(lib, kw, status):
    assert linear(lib, **kw) == status


def test_linear_workspace(lib):
    f = lib.linear_int4_rows_workspace_bytes
    assert f(0, 8, 64) == 0 and f(4, 8, 40) == 0
    split = [(M, N, K) for M in (1, 33, 100) for N in (16, 300) for K in (8192, 65536) if f(M, N, K)]
    assert split                                      # long sums over few tiles are split
    for M, N, K in split:
        need = f(M, N, K)
        assert need % 256 == 0
        kw = dict(M=M, N=N, K=K, cs=K, ldo=N, rs=N)
        assert linear(lib, nb=need - 1, **kw) == EWORKSPACE
        assert linear(lib, ws=0, **kw) == EINVAL
        assert linear(lib, ws=A + 16, **kw) == EALIGN


NAMES = ("history", "n_history", "history_offsets", "n_prompt", "repetition", "frequency", "presence", "bias_ids",
         "bias_values", "n_bias", "bias_offsets", "mask", "n_masks", "mask_stride", "mask_index")
GOOD = dict(history=A, n_history=10, history_offsets=A, n_prompt=A, repetition=A, frequency=A, presence=A, bias_ids=A,
            bias_values=A, n_bias=3, bias_offsets=A, mask=A, n_masks=8, mask_stride=4, mask_index=A)


def rules(**kw):
    r = {**GOOD, **kw}
    return binding._RULES.pack(*(r[n] for n in NAMES))


def apply(lib, x=A, xs=100, dt=2, d=A, R=2, T=4, V=100, r=None, out=A, ldo=100):
    return lib.logit_rules_apply(x, xs, dt, d, R, T, V, rules() if r is None else r, out, ldo, None)


def verify(lib, x=A, xs=100, dt=2, d=A, dp=A, un=A, R=2, T=4, V=100, r=None, k=4, tau=1.0, lmax=A, amax=A, tid=A,
           tlog=A, lse=A, p=A, n=A, ws=A, nb=1 << 30):
    return lib.logit_rules_verify(x, xs, dt, d, dp, un, R, T, V, rules() if r is None else r, k, tau, lmax, amax, tid,
                                  tlog, lse, p, n, ws, nb, None)


ROWS = [(dict(R=0), EINVAL), (dict(T=0), EINVAL), (dict(T=17), EINVAL), (dict(R=257, T=16), EINVAL),
        (dict(V=0), EINVAL), (dict(dt=4), EINVAL), (dict(x=0), EINVAL), (dict(d=0), EINVAL), (dict(xs=99), EINVAL),
        (dict(x=A + 2), EALIGN), (dict(d=A + 1), EALIGN)]
BAD_RULES = [(dict(n_history=-1), EINVAL), (dict(history=0), EINVAL), (dict(history_offsets=0), EINVAL),
             (dict(n_bias=-1), EINVAL), (dict(bias_ids=0), EINVAL), (dict(bias_values=0), EINVAL),
             (dict(bias_offsets=0), EINVAL), (dict(n_masks=0), EINVAL), (dict(mask_stride=3), EINVAL),
             (dict(mask_index=0, n_masks=7), EINVAL), (dict(mask=0), EINVAL), (dict(history=A + 2), EALIGN),
             (dict(history_offsets=A + 4), EALIGN), (dict(n_prompt=A + 1), EALIGN), (dict(repetition=A + 2), EALIGN),
             (dict(frequency=A + 2), EALIGN), (dict(presence=A + 2), EALIGN), (dict(bias_ids=A + 2), EALIGN),
             (dict(bias_values=A + 2), EALIGN), (dict(bias_offsets=A + 4), EALIGN), (dict(mask=A + 2), EALIGN),
             (dict(mask_index=A + 2), EALIGN)]


@pytest.mark.parametrize("call", [apply, verify])
def test_rules_refusals(lib, call):
    for kw, status in ROWS:
        assert call(lib, **kw) == status, kw
    for kw, status in BAD_RULES:
        assert call(lib, r=rules(**kw)) == status, kw
    big = (1 << 24) + 1
    r = rules(mask_stride=1 << 20)
    assert (call(lib, V=big, xs=big, r=r) if call is verify else call(lib, V=big, xs=big, r=r, ldo=big)) == EUNSUPPORTED


def test_apply_refusals(lib):
    assert apply(lib, out=0) == EINVAL
    assert apply(lib, ldo=99) == EINVAL
    assert apply(lib, out=A + 2) == EALIGN


@pytest.mark.parametrize("kw,status", [
    (dict(k=-1), EINVAL), (dict(k=17), EINVAL), (dict(V=3, xs=3), EINVAL), (dict(tau=0.0), EINVAL),
    (dict(tau=-1.0), EINVAL), (dict(tau=math.inf), EINVAL), (dict(tau=math.nan), EINVAL), (dict(dp=0), EINVAL),
    (dict(un=0), EINVAL), (dict(p=0), EINVAL), (dict(lmax=0), EINVAL), (dict(amax=0), EINVAL), (dict(tid=0), EINVAL),
    (dict(tlog=0), EINVAL), (dict(n=0), EINVAL), (dict(ws=0), EINVAL), (dict(ws=A + 64), EALIGN),
    (dict(nb=1000), EWORKSPACE), (dict(lse=A + 2), EALIGN), (dict(n=A + 2), EALIGN), (dict(dp=A + 2), EALIGN),
])
def test_verify_refusals(lib, kw, status):
    assert verify(lib, **kw) == status


def ruled(lib, h=A, w=A, s=A, d=A, dp=A, un=A, R=2, T=4, V=100, H=64, r=None, k=4, tau=1.0, ws=A, nb=1 << 30, n=A):
    return lib.verify_lm_head_int4_ruled(h, w, s, d, dp, un, R, T, V, H, rules() if r is None else r, k, tau, A, A, A,
                                         A, A, A, n, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(R=0), EINVAL), (dict(T=17), EINVAL), (dict(R=2000, T=3), EINVAL), (dict(H=16), EINVAL), (dict(H=48), EINVAL),
    (dict(h=0), EINVAL), (dict(w=0), EINVAL), (dict(s=0), EINVAL), (dict(d=0), EINVAL), (dict(ws=0), EINVAL),
    (dict(k=17), EINVAL), (dict(tau=0.0), EINVAL), (dict(un=0), EINVAL), (dict(n=0), EINVAL), (dict(nb=4096), EWORKSPACE),
    (dict(ws=A + 16), EALIGN), (dict(h=A + 8), EALIGN), (dict(w=A + 8), EALIGN), (dict(H=8224), EUNSUPPORTED),
    (dict(r=rules(bias_values=0)), EINVAL), (dict(r=rules(mask=A + 1)), EALIGN),
])
def test_ruled_refusals(lib, kw, status):
    assert ruled(lib, **kw) == status


def test_workspace_sizes(lib):
    f, g = lib.logit_rules_verify_workspace_bytes, lib.verify_lm_head_int4_ruled_workspace_bytes
    assert f(0, 1, 10, 0) == 0 and f(1, 17, 10, 0) == 0 and f(1, 1, 10, 11) == 0 and f(1, 1, 10, 17) == 0
    assert f(1, 1, (1 << 24) + 1, 0) == 0
    assert f(64, 4, 151936, 16) % 256 == 0
    assert g(64, 4, 151936, 5120, 16) >= 256 * 151936 * 4 + f(64, 4, 151936, 16) + lib.verify_lm_head_int4_workspace_bytes(64, 4, 151936, 5120)
    assert g(64, 4, 151936, 48, 16) == 0


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(2, 64, dtype=torch.float16), torch.ones(64, dtype=torch.float16)
    with pytest.raises(TypeError):
        binding.rms_norm(x, w)
    with pytest.raises(TypeError):
        binding.rms_norm_int8(x, w)
    with pytest.raises(TypeError):
        binding.quantize_rows(x)
    with pytest.raises(TypeError):
        binding.linear_int4(torch.zeros(2, 64, dtype=torch.int8), torch.ones(2), torch.zeros(8, 32, dtype=torch.uint8))
    with pytest.raises(TypeError):
        binding.LogitRules(repetition=torch.ones(2))
    with pytest.raises(TypeError):
        binding.apply_logit_rules(torch.zeros(2, 10), None, R=2)
    with pytest.raises(TypeError):
        binding.verify_logits(torch.zeros(2, 10), None, R=2)
    assert binding.LogitRules().packed == bytes(ctypes.sizeof(ctypes.c_int64) * 15)
