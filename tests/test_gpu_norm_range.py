"""Rows whose sum of squares leaves binary32, next to ordinary ones (GPU).
The tolerances are those of test_gpu_norm: the scale of such a row's sum is a
power of two, which rounds nothing."""
import pytest
import torch

from tests.test_gpu_norm import DT, close_codes, close_norm, gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


# the sum of 8192 squares overflows from an rms of 2^57.5 = 2.0e17 on
LARGE = [2.0 ** 57, 1.9e17, 2.1e17, 3e17, 1e18, 1e25, 1e30, 1e37]
# without eps: below 2^-40 the sum is taken at another scale; squares are
# subnormal from 2^-63 on and gone below 2^-75; bfloat16 and binary32 rows go
# down to subnormal numbers themselves
SMALL = [2.0 ** -39, 2.0 ** -41, 1e-18, 2.0 ** -70, 1e-25, 1e-36, 1e-40]


def rows(dt, H, sizes, seed):
    """Rows of those sizes in turn, ordinary ones between them."""
    g = torch.Generator().manual_seed(seed)
    n = torch.randn(3 * len(sizes), H, generator=g).clamp(-4, 4)
    for i, s in enumerate(sizes):
        n[3 * i] *= s
        n[3 * i][torch.rand(H, generator=g) < 0.2] = s          # some of them constant in part
        n[3 * i, 0] = s
    return n.to(dt)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [1, 8, 77, 512, 5120, 8192])
@pytest.mark.parametrize("sizes,eps", [(LARGE, 1e-6), (LARGE, 0.0), (SMALL, 0.0), (LARGE, 3e38), (SMALL, 1e-30)])
def test_norm(b, H, dt, sizes, eps):
    x = rows(DT[dt], H, sizes, H)
    w = (1 + 0.3 * torch.randn(H, generator=torch.Generator().manual_seed(1))).to(DT[dt])
    for r in (None, x / 4):
        for odt in (torch.float32, torch.bfloat16):
            got = b.rms_norm(gpu(x), gpu(w), gpu(r), eps=eps, out_dtype=odt)
            close_norm(got if r is None else got[0], x, w, r, eps)
        c = torch.full((H,), 0.5, dtype=torch.float16)
        got = b.rms_norm_int8(gpu(x), gpu(w), gpu(r), channel_scales=gpu(c), eps=eps)
        # rows whose peak is below 2^-100 have codes and a scale of 0
        t = (x.double() + (0 if r is None else r.double())).abs().mul(w.double().abs() * 0.5).amax(dim=1)
        live = t > 2.0 ** -99
        close_codes(got[0][live.cuda()], got[1][live.cuda()], x[live], w, None if r is None else r[live], c, eps)
        dead = (t < 2.0 ** -101).cuda()
        assert int(got[0][dead].abs().sum()) == 0 and float(got[1][dead].abs().sum()) == 0


@pytest.mark.parametrize("size", [1e30, 1e-30])
def test_many_rows_of_which_some_are_far_off(b, size):
    """More rows than workgroups: such rows behind each other and behind
    ordinary ones in one workgroup."""
    M, H = 5000, 4100
    g = torch.Generator().manual_seed(3)
    x = torch.randn(M, H, generator=g)
    x[torch.rand(M, generator=g) < 0.4] *= size
    w = 1 + 0.3 * torch.randn(H, generator=g)
    close_norm(b.rms_norm(gpu(x), gpu(w), eps=0.0, out_dtype=torch.float32), x, w, None, 0.0)
    q, s = b.rms_norm_int8(gpu(x), gpu(w), eps=0.0)
    close_codes(q, s, x, w, None, None, 0.0)


def test_large_and_small_channels_in_one_row(b):
    """The small channels of a large row, and the large weights of a small one,
    keep their bits."""
    H = 600
    x = torch.full((3, H), 1e30)
    x[0, 1::2] = 1e-6
    x[1] = 3e38
    x[1, 7] = 2.0 ** 10
    x[2] = 1e-26
    x[2, ::3] = 2.0 ** -140
    w = torch.ones(H)
    w[5], w[6], w[7], w[9] = 1e30, 1e-12, 1e20, 1e25
    close_norm(b.rms_norm(gpu(x), gpu(w), eps=0.0, out_dtype=torch.float32), x, w, None, 0.0)
    q, s = b.rms_norm_int8(gpu(x[2:]), gpu(w), eps=0.0)
    close_codes(q, s, x[2:], w, None, None, 0.0)


def test_rows_without_a_finite_norm_stay_as_they_were(b):
    H = 300
    x = torch.ones(4, H)
    x[0, 3], x[1, 4], x[2] = float("inf"), float("nan"), 0
    y = b.rms_norm(gpu(x), torch.ones(H, device="cuda"), eps=0.0, out_dtype=torch.float32).cpu()
    assert torch.isnan(y[0, 3]) and torch.equal(y[0, 4:], torch.zeros(H - 4))
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all() and torch.equal(y[3], torch.ones(H))
    q, s = (t.cpu() for t in b.rms_norm_int8(gpu(x), torch.ones(H, device="cuda"), eps=0.0))
    assert int(q[:3].abs().sum()) == 0 and not torch.isfinite(s[0]) and torch.isnan(s[1]) and s[2] == 0


@pytest.mark.parametrize("H", [1, 5120, 8192])
def test_binary16_rows_at_their_ends(b, H):
    """Their squares' sums lie between 2^-48 and 2^47: no other scale is needed."""
    x = torch.zeros(4, H)
    x[0], x[1], x[2, -1], x[3] = 65504, 2.0 ** -24, 2.0 ** -24, -65504
    x, w = x.half(), torch.ones(H, dtype=torch.float16)
    for r in (None, x):
        got = b.rms_norm(gpu(x), gpu(w), gpu(r), eps=0.0, out_dtype=torch.float32)
        close_norm(got if r is None else got[0], x, w, r, 0.0)
        got = b.rms_norm_int8(gpu(x), gpu(w), gpu(r), eps=0.0)
        close_codes(got[0], got[1], x, w, r, None, 0.0)
