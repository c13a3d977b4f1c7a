"""The gelu of the linear layer's epilogue over its whole range (GPU), against
y / 2 * erfc(-y / sqrt(2)) in 64 bits and relative to the value itself.

Tolerance, u = 2^-24: the exponent y^2 / 2 carries 3 u (square, constant,
product); the fitted factor 0.34 u and below 4 u for its evaluation, its
argument 3 u (sum, reciprocal), exp2 2 u, four products and a difference at
most 4 u: (1.5 y^2 + 14) u, then half a step of the output's type.  Where exp2
is subnormal it is off by 2^-150, times at most |y| + 1; then half of the
type's smallest step."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_linear import DT, SMALLEST, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def want64(y):
    return 0.5 * y * np.vectorize(math.erfc, otypes=[np.float64])(-y * math.sqrt(0.5))


# the stream, its split sum, tiles of 32 rows, with a split sum, of 64 and 128
@pytest.mark.parametrize("M,K", [(1, 32), (16, 32), (3, 16384), (20, 64), (40, 8192), (1100, 64), (2100, 32)])
@pytest.mark.parametrize("dt", list(DT))
def test_gelu(b, M, K, dt):
    dt = DT[dt]
    for N in (5003, 5004):                             # N % 4 picks another epilogue
        y = torch.cat((torch.linspace(-14.4, 8.0, N - 3), torch.tensor([0.0, -0.0, 1e-30]))).to(dt)
        codes = torch.zeros(M, K, dtype=torch.int8, device="cuda")
        packed = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
        got = b.linear_int4(codes, torch.ones(M, device="cuda"), packed, bias=y.cuda(), activation="gelu", out_dtype=dt)
        assert torch.equal(got, got[:1].expand(M, N))
        y64 = y.double().numpy()
        z = want64(y64)
        half = torch.finfo(dt).eps / 2
        rel = (1.5 * y64 ** 2 + 14) * U
        tol = np.abs(z) * (rel + half * (1 + rel)) + 2.0 ** -150 * (np.abs(y64) + 1) + SMALLEST[dt] / 2
        off = np.abs(got[0].double().cpu().numpy() - z)
        assert np.all(off <= tol), (float((off / tol).max()), y64[(off / tol).argmax()])


def test_gelu_far_out(b):
    y = torch.tensor([-1e30, -3e38, -40.0, 40.0, 1e30, 3e38, math.inf, -math.inf, math.nan])
    N = y.numel()
    for M in (2, 40):
        got = b.linear_int4(torch.zeros(M, 64, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda"),
                            torch.zeros(N, 32, dtype=torch.uint8, device="cuda"), bias=y.cuda(), activation="gelu",
                            out_dtype=torch.float32).cpu()
        for r in got:
            assert r[:3].tolist() == [0.0] * 3 and r[3:7].tolist() == y[3:7].tolist() and torch.isnan(r[7:]).all()
