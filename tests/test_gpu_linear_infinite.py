"""Row scales that are infinite or NaN, on sums of either sign and of 0 (GPU):
what the epilogue's formulas make of them, on every kernel."""
import numpy as np
import pytest
import torch

from int4_output_head_amd import synth

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


# the sums' signs -1, 0, 1 under row scales inf, -inf and NaN
WANT = {None: ([-INF, NAN, INF], [INF, NAN, -INF]), "relu": ([0.0, NAN, INF], [INF, NAN, 0.0]),
        "gelu": ([NAN, NAN, INF], [INF, NAN, NAN]), "silu": ([NAN, NAN, INF], [INF, NAN, NAN])}


@pytest.mark.parametrize("act", list(WANT))
@pytest.mark.parametrize("M,N,K", [(4, 9, 64), (5, 300, 16384), (20, 300, 8192), (40, 302, 96), (1100, 5000, 32),
                                   (2100, 5000, 32)])
def test_infinite_row_scales(b, M, N, K, act):
    q = np.zeros((N, K), np.int8)
    q[:, 0] = np.arange(N) % 3 - 1
    codes = np.zeros((M, K), np.int8)
    codes[:, 0] = 3
    rs = torch.ones(M)
    rs[0], rs[1], rs[2] = INF, -INF, NAN
    packed = torch.from_numpy(synth.pack_int4(q)).cuda()
    for bias in (None, torch.full((N,), 0.25, device="cuda")):
        got = b.linear_int4(torch.from_numpy(codes).cuda(), rs.cuda(), packed, activation=act, bias=bias,
                            out_dtype=torch.float32).cpu().numpy()
        for row, want in zip(got[:2], WANT[act]):
            assert np.array_equal(row, np.resize(np.float32(want), N), equal_nan=True)
        assert np.isnan(got[2]).all() and np.isfinite(got[3:]).all()
        assert np.array_equal(got[3:], np.tile(got[3], (M - 3, 1)))
