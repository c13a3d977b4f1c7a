"""The norm and the 8-bit rows against their formulas in 64 bits (GPU).

Tolerances, u = 2^-24 the binary32 half step.  rstd: each term of the sum of
squares is rounded at most 48 times on its way (16 sums in a thread, 6 across
lanes, 16 across waves, its own product and operands), which the root halves:
24 u, and 4 u for the division, eps, root and reciprocal.  normed: 28 u + 1 u
(h) + 2 u (two products) < 32 u, then half a step of the output's type, or half
of the type's smallest step.  8 bits: t carries 3 u, the peak 3 u, 127 / peak
and the last product 2 u: 8 u of at most 127 steps beyond the half step of the
rounding; row_scale 3 + 28 + 2 < 34 u."""
import numpy as np
import pytest
import torch

from oracle import rows

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def make(M, H, dt, seed, residual=True, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    spread = torch.exp(0.7 * torch.randn(H, generator=g))
    x = (scale * torch.randn(M, H, generator=g) * spread).to(dt)
    r = (3 * scale * torch.randn(M, H, generator=g) * spread).to(dt) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(dt)
    c = torch.exp(-4 + 0.5 * torch.randn(H, generator=g)).to(torch.float16)
    return x, r, w, c


def f64(t):
    return None if t is None else t.double().numpy()


def f32(t):
    return None if t is None else t.float().numpy()


def gpu(t):
    return None if t is None else t.cuda()


def close_norm(got, x, w, r, eps):
    want = rows.norm64(f64(x), f64(w), f64(r), eps)
    half = torch.finfo(got.dtype).eps / 2
    tol = np.abs(want) * (half * (1 + 32 * U) + 32 * U) + SMALLEST[got.dtype] / 2
    off = np.abs(f64(got.cpu()) - want)
    assert np.all(off <= tol), float((off / tol).max())


def close_codes(codes, row_scales, x, w, r, c, eps, norm=True):
    codes, row_scales = codes.cpu().numpy(), row_scales.cpu().double().numpy()
    t = rows.scaled64(f64(x), f64(w), f64(r), f64(c))
    peak = np.abs(t).max(axis=1, keepdims=True)
    ideal = t * 127 / peak
    assert np.all(np.abs(codes - ideal) <= 0.5 + 127 * 8 * U)
    # bit for bit in the documented order
    assert np.array_equal(codes, rows.codes32(f32(x), f32(w), f32(r), f32(c)))
    want = peak[:, 0] / 127 * (rows.rstd64(rows.add64(f64(x), f64(r)), eps)[:, 0] if norm else 1.0)
    assert np.all(np.abs(row_scales - want) <= 34 * U * want)


SHAPES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 31), (1, 5120), (16, 5120), (17, 512), (4, 8192), (3, 8185), (2, 4097),
          (1300, 257), (2500, 96), (1030, 5121), (1100, 8192)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,H", SHAPES)
def test_norm(b, M, H, dt):
    for residual in (False, True):
        x, r, w, _ = make(M, H, DT[dt], 7 * M + H, residual)
        for odt in (torch.float16, torch.bfloat16, torch.float32):
            got = b.rms_norm(gpu(x), gpu(w), gpu(r), eps=1e-5, out_dtype=odt)
            if residual:
                got, total = got
                # one rounding of the binary32 sum
                assert torch.equal(total.cpu(), (x.float() + r.float()).to(x.dtype))
            assert got.shape == x.shape and got.dtype == odt
            close_norm(got, x, w, r, 1e-5)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,H", SHAPES)
def test_norm_int8(b, M, H, dt):
    for residual, channel in ((True, True), (False, True), (True, False)):
        x, r, w, c = make(M, H, DT[dt], 3 * M + H, residual)
        c = c if channel else None
        got = b.rms_norm_int8(gpu(x), gpu(w), gpu(r), channel_scales=gpu(c), eps=1e-6)
        close_codes(got[0], got[1], x, w, r, c, 1e-6)
        if residual:
            assert torch.equal(got[2].cpu(), (x.float() + r.float()).to(x.dtype))
        q = b.quantize_rows(gpu(x), channel_scales=gpu(c))
        close_codes(q[0], q[1], x, None, None, c, 0.0, norm=False)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,H", [(1, 8193), (3, 9000), (2, 16384), (1, 16385), (5, 25600), (2, 32769), (1, 65536),
                                 (1100, 8200)])
def test_long_rows_in_8_bits(b, M, H, dt):
    for channel in (True, False):
        x, _, _, c = make(M, H, DT[dt], M + H, False)
        x[:, -1] *= 50                                 # the peak in the overlapping chunks of some rows
        c = c if channel else None
        q, sc = b.quantize_rows(gpu(x), channel_scales=gpu(c))
        close_codes(q, sc, x, None, None, c, 0.0, norm=False)
        buf = torch.full((M, H + 3), 7, dtype=DT[dt])  # strided, unaligned rows
        buf[:, 3:] = x
        q2, sc2 = b.quantize_rows(gpu(buf)[:, 3:], channel_scales=gpu(c))
        assert torch.equal(q, q2) and torch.equal(sc, sc2)


def test_long_zero_tiny_and_non_finite_rows(b):
    H = 20001
    x = torch.ones(6, H)
    x[0], x[1] = 0, 2.0 ** -110
    x[2, 20000], x[3, 5], x[4, 12000] = float("inf"), float("nan"), -float("inf")
    q, s = b.quantize_rows(x.cuda())
    assert torch.equal(q[:5].cpu(), torch.zeros(5, H, dtype=torch.int8))
    s = s.cpu()
    assert s[0] == 0 and s[1] == 0 and torch.isinf(s[2]) and torch.isnan(s[3]) and torch.isinf(s[4])
    assert torch.equal(q[5].cpu(), torch.full((H,), 127, dtype=torch.int8))


def test_weights_of_another_type(b):
    x, r, w, c = make(9, 1000, torch.bfloat16, 5)
    for wd in DT.values():
        close_norm(b.rms_norm(gpu(x), gpu(w.to(wd)), gpu(r))[0], x, w.to(wd), r, 1e-6)


def test_strided_and_misaligned_rows(b):
    for H, lead, off in ((256, 300, 3), (1001, 1003, 1), (64, 64, 5)):
        g = torch.Generator().manual_seed(H)
        big = torch.randn(7 * lead + off + H, generator=g).to(torch.float16).cuda()
        x = torch.as_strided(big, (7, H), (lead, 1), off)
        w = torch.randn(H + 1, generator=g).to(torch.float16).cuda()[1:]
        r = torch.randn(7, H + 5, generator=g).to(torch.float16).cuda()[:, 2: 2 + H]
        out, total = b.rms_norm(x, w, r)
        close_norm(out, x.cpu(), w.cpu(), r.cpu(), 1e-6)
        assert torch.equal(total.cpu(), (x.float() + r.float()).half().cpu())
        q, s = b.quantize_rows(x)
        close_codes(q, s, x.cpu(), None, None, None, 0.0, norm=False)
    with pytest.raises(ValueError):
        b.rms_norm(torch.zeros(4, 8, dtype=torch.float16, device="cuda").t(), torch.ones(4, dtype=torch.float16, device="cuda"))


def test_leading_dims_and_sum_in_place(b):
    x, r, w, _ = make(12, 640, torch.bfloat16, 1)
    a = b.rms_norm(gpu(x).view(3, 4, 640), gpu(w), gpu(r).view(3, 4, 640))
    assert a[0].shape == (3, 4, 640)
    close_norm(a[0].view(12, 640), x, w, r, 1e-6)
    # the C entry point writes the sum over x or over the residual
    for which in (0, 1):
        xc, rc = gpu(x), gpu(r)
        out = torch.empty(12, 640, dtype=torch.float16, device="cuda")
        st = b.load_library().rms_norm_rows(xc.data_ptr(), 640, rc.data_ptr(), 640, 1, gpu(w).data_ptr(), 1, 12, 640,
                                            1e-6, (xc, rc)[which].data_ptr(), out.data_ptr(), 0,
                                            torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert torch.equal((xc, rc)[which].cpu(), a[1].view(12, 640).cpu())
        assert torch.equal((xc, rc)[1 - which].cpu(), (r, x)[which])
        assert torch.equal(out, a[0].view(12, 640))


def test_zero_tiny_and_non_finite_rows(b):
    H = 200
    x = torch.ones(6, H, dtype=torch.float32)
    x[0] = 0
    x[1] = 2.0 ** -110
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    w = torch.ones(H)
    y = b.rms_norm(x.cuda(), w.cuda(), eps=1e-6, out_dtype=torch.float32).cpu()
    assert torch.equal(y[0], torch.zeros(H))
    assert torch.isnan(y[2]).all()
    assert torch.isnan(y[3, 7]) and torch.equal(y[3, :7], torch.zeros(7))
    assert torch.allclose(y[4], torch.full((H,), 1 / np.sqrt(1 + 1e-6).item()), rtol=1e-6)
    for got in (b.rms_norm_int8(x.cuda(), w.cuda()), b.quantize_rows(x.cuda())):
        q, s = got[0].cpu(), got[1].cpu()
        assert torch.equal(q[:4], torch.zeros(4, H, dtype=torch.int8))
        assert s[0] == 0 and s[1] == 0 and torch.isnan(s[2]) and not torch.isfinite(s[3])
        assert torch.equal(q[4:], torch.full((2, H), 127, dtype=torch.int8))


def test_a_row_gives_the_same_bits_in_every_batch_of_its_shape(b):
    x, r, w, c = make(40, 5120, torch.float16, 9)
    whole = b.rms_norm_int8(gpu(x), gpu(w), gpu(r), channel_scales=gpu(c))
    one = b.rms_norm_int8(gpu(x[7:8]), gpu(w), gpu(r[7:8]), channel_scales=gpu(c))
    for u, v in zip(whole, one):
        assert torch.equal(u[7:8], v)


def test_streams_and_graph(b):
    x, r, w, c = make(64, 5120, torch.float16, 2)
    X, Rr, W, C = map(gpu, (x, r, w, c))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = b.rms_norm(X, W, Rr)
    side.synchronize()
    assert torch.equal(on_side[0], b.rms_norm(X, W, Rr)[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = b.rms_norm(X, W, Rr) + b.rms_norm_int8(X, W, Rr, channel_scales=C)
    for k in range(3):
        X.copy_(make(64, 5120, torch.float16, 50 + k)[0])
        want = b.rms_norm(X, W, Rr) + b.rms_norm_int8(X, W, Rr, channel_scales=C)
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip(out, want):
            assert torch.equal(u, v)


def test_refusals(b):
    x, r, w, c = (gpu(t) for t in make(4, 64, torch.float16, 0))
    for bad in (lambda: b.rms_norm(x, w[:63]), lambda: b.rms_norm(x, w, r[:3]), lambda: b.rms_norm(x, w, r.bfloat16()),
                lambda: b.rms_norm_int8(x, w, channel_scales=c[:10]), lambda: b.rms_norm(x[:0], w),
                lambda: b.rms_norm(x.expand(2, 4, 64), w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: b.rms_norm(x.int(), w), lambda: b.rms_norm(x, w, out_dtype=torch.int8),
                lambda: b.quantize_rows(x, channel_scales=c.float()), lambda: b.rms_norm(x, w.cpu())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(RuntimeError):
        b.rms_norm(x, w, eps=-1.0)
    big = torch.zeros(1, 8193, dtype=torch.float16, device="cuda")
    with pytest.raises(RuntimeError):
        b.rms_norm(big, big[0])
