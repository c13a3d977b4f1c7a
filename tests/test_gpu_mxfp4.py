"""Rows in microscaled 4-bit floating point, and products of two such matrices
(GPU).

The quantisation and the values are bit for bit the oracle's.  Products whose
sums are whole numbers of quarters below 2^24 are exact in binary32 in any
order, so they have to equal the 64-bit product.  Otherwise, with u = 2^-24 and
S the sum of the products' magnitudes: at most K additions, each off by no more
than a whole step (2 u) of a partial sum that is at most S: 2 K u S; + bias u |y|;
the activation's slope at most 1.13 and its own 8 u |y| ((1.5 y^2 + 14) u |z| for the
gelu); u (|z| + |residual|) for the last sum, then half a step of the output's
type or half of its smallest step."""
import numpy as np
import pytest
import torch

from oracle import mxfp4

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def same_codes(b, x):
    codes, scales = b.quantize_mxfp4(x.cuda())
    want_codes, want_scales = mxfp4.quantize(x.double().numpy().reshape(-1, x.shape[-1]))
    H = x.shape[-1]
    assert codes.shape == x.shape[:-1] + (H // 2,) and scales.shape == x.shape[:-1] + (H // 32,)
    assert np.array_equal(scales.cpu().numpy().reshape(-1, H // 32), want_scales)
    assert np.array_equal(codes.cpu().numpy().reshape(-1, H // 2), want_codes)
    return codes, scales


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,H", [(1, 32), (1, 65536), (3, 96), (7, 5120), (130, 2080), (4099, 64), (2, 8192)])
def test_quantize(b, M, H, dt):
    g = torch.Generator().manual_seed(M + H)
    x = torch.randn(M, H, generator=g) * torch.exp2(torch.randint(-9, 9, (M, H), generator=g).float())
    codes, scales = same_codes(b, x.to(DT[dt]))
    for odt in DT.values():
        got = b.dequantize_mxfp4(codes, scales, out_dtype=odt)
        want = torch.from_numpy(mxfp4.values(codes.cpu().numpy(), scales.cpu().numpy())).to(odt)
        assert got.dtype == odt and torch.equal(got.cpu(), want)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_every_16_bit_value(b, dt):
    """All bit patterns, each beside peaks that give it several scales."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(DT[dt])
    bits = bits[bits.isfinite()]
    x = torch.zeros(len(bits), 64, dtype=DT[dt])
    x[:, 0] = bits
    x[:, 32] = bits
    x[:, 33] = bits * 3
    x[:, 34] = bits.abs().clamp(min=2.0 ** -14) * torch.where(torch.arange(len(bits)) % 2 == 0, 1.5, 4.0)
    x = torch.where(x.isfinite(), x, torch.zeros((), dtype=DT[dt]))
    same_codes(b, x)


def test_binary32_ends(b):
    """Ties, neighbours of every border, subnormal and largest numbers."""
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.9999995], np.float32)
    near = np.concatenate([borders, np.nextafter(borders, 0, dtype=np.float32),
                           np.nextafter(borders, 8, dtype=np.float32), np.zeros(4, np.float32)])[None]
    near = np.concatenate([near, -near], axis=1)
    x = np.zeros((1, 32 * 8), np.float32)
    rows = []
    for e in (-149, -140, -130, -127, -126, -125, -124, -100, -1, 0, 1, 60, 120, 124, 125):
        x = np.zeros((near.shape[1], 32), np.float32)
        with np.errstate(all="ignore"):
            x[:, 0] = np.ldexp(np.float32(4.0), e)
            x[:, 1] = np.ldexp(near[0], e)
            x[:, 2] = np.ldexp(near[0][::-1], e - 1)
            x[:, 31] = np.ldexp(np.float32(1.5), e - 20)
        rows.append(np.where(np.isfinite(x), x, np.float32(3.4028235e38)))
    same_codes(b, torch.from_numpy(np.concatenate(rows)))


def test_bad_values_stay_in_their_32_channels(b):
    x = torch.randn(5, 96)
    x[1, 40], x[2, 0], x[3, 95] = float("nan"), float("inf"), -float("inf")
    codes, scales = same_codes(b, x)
    v = b.dequantize_mxfp4(codes, scales, out_dtype=torch.float32).cpu()
    assert v[1, 32:64].isnan().all() and v[2, :32].isnan().all() and v[3, 64:].isnan().all()
    assert v.isnan().sum() == 96
    y = b.linear_mxfp4(codes, scales, *b.quantize_mxfp4(torch.randn(20, 96).cuda()), out_dtype=torch.float32).cpu()
    assert y[1:4].isnan().all() and y[0].isfinite().all() and y[4].isfinite().all()
    y = b.linear_mxfp4(*b.quantize_mxfp4(torch.randn(40, 96).cuda()), codes, scales, out_dtype=torch.float32).cpu()
    assert y[:, 1:4].isnan().all() and y[:, 0].isfinite().all() and y[:, 4].isfinite().all()


def test_strided_rows(b):
    wide = torch.randn(9, 200).to(torch.bfloat16).cuda()
    for at in (0, 1, 3):
        got = b.quantize_mxfp4(wide[:, at:at + 160])
        want = b.quantize_mxfp4(wide[:, at:at + 160].contiguous())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x = torch.randn(70000, 32).to(torch.float16).cuda()[::1]
    tall = torch.zeros(70000, 40, dtype=torch.float16, device="cuda")
    tall[:, :32] = x
    got, want = b.quantize_mxfp4(tall[:, :32]), b.quantize_mxfp4(x)     # more rows than a grid is high
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---------------------------------------------------------------- products

def exact(M, N, K, seed):
    """Codes and scales whose products' sums are quarters below 2^24."""
    g = np.random.default_rng(seed)
    c = lambda n: torch.from_numpy(g.integers(0, 256, (n, K // 2), dtype=np.uint8))  # noqa: E731
    s = lambda n: torch.from_numpy(g.integers(127, 129, (n, K // 32), dtype=np.uint8))  # noqa: E731
    return c(M), s(M), c(N), s(N)


def rough(M, N, K, seed, dt):
    g = torch.Generator().manual_seed(seed)
    t = lambda n: tuple(torch.from_numpy(v) for v in mxfp4.quantize(  # noqa: E731
        (torch.randn(n, K, generator=g) * torch.exp(torch.randn(K, generator=g))).numpy()))
    return (*t(M), *t(N)), (0.5 * torch.randn(N, generator=g)).to(dt), torch.randn(M, N, generator=g).to(dt)


def check(got, args, act=None, bias=None, residual=None):
    K = 2 * args[0].shape[1]
    f = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    z, y, S = mxfp4.linear64(*(t.numpy() for t in args), f(bias), act, f(residual))
    own = 0.0
    if act == "silu":
        own = 8 * U * np.abs(y)
    elif act == "gelu":
        own = (1.5 * y * y + 14) * U * np.abs(z if residual is None else z - f(residual))
    tol = 1.13 * (2 * K * U * S + U * np.abs(y)) + own
    if residual is not None:
        tol = tol + U * (np.abs(z) + np.abs(f(residual)) + tol)
    tol = tol + torch.finfo(got.dtype).eps / 2 * (np.abs(z) + tol) + SMALLEST[got.dtype] / 2
    off = np.abs(got.cpu().double().numpy() - z)
    assert np.all(off <= tol), float((off / tol).max())


# one row to many, odd widths, K in all its remainders of 128 and 512, split sums
SHAPES = [(1, 1, 32), (1, 16, 64), (1, 5120, 5120), (3, 17, 96), (16, 512, 5120), (16, 100, 8192), (16, 3, 8224),
          (17, 333, 2048), (2, 40, 20480), (32, 64, 1024), (32, 1000, 8192), (20, 33, 20480), (33, 65, 160),
          (33, 2, 64), (64, 128, 128), (50, 300, 4096), (65, 129, 352), (128, 256, 1024), (200, 127, 8192),
          (300, 513, 640), (257, 1030, 512), (1000, 100, 2080), (130, 3, 64), (2100, 2600, 32), (4096, 4097, 64),
          (2049, 2305, 544), (700, 5120, 1536), (512, 18992, 96)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_exact_products(b, M, N, K):
    args = exact(M, N, K, M + N + K)
    got = b.linear_mxfp4(*(t.cuda() for t in args), out_dtype=torch.float32)
    want = torch.from_numpy(mxfp4.values(*(t.numpy() for t in args[:2]))).cuda() @ \
        torch.from_numpy(mxfp4.values(*(t.numpy() for t in args[2:]))).cuda().T.contiguous()
    assert want.abs().max() < 2 ** 22
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("K", [32, 992, 1024, 1056, 2080, 2944, 3616, 4064, 4096, 4640, 5632, 6112, 6144, 6176, 7200, 8160])
@pytest.mark.parametrize("M,N", [(1, 9000), (7, 37), (16, 8200)])
def test_exact_products_of_few_rows(b, M, N, K):
    """Every number of steps per wave, and more tiles than workgroups."""
    args = exact(M, N, K, M + N + K)
    got = b.linear_mxfp4(*(t.cuda() for t in args), out_dtype=torch.float32)
    want = torch.from_numpy(mxfp4.values(*(t.numpy() for t in args[:2]))).cuda() @ \
        torch.from_numpy(mxfp4.values(*(t.numpy() for t in args[2:]))).cuda().T.contiguous()
    assert want.abs().max() < 2 ** 22
    assert torch.equal(got.double(), want)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("act", [None, "relu", "gelu", "silu"])
@pytest.mark.parametrize("M,N,K", [(5, 70, 256), (40, 72, 256), (150, 131, 4096), (260, 300, 96), (900, 644, 512)])
def test_epilogue(b, M, N, K, act, dt):
    args, bias, residual = rough(M, N, K, M + len(dt), DT[dt])
    dev = [t.cuda() for t in args]
    for bi, re in ((bias, residual), (bias, None), (None, residual), (None, None)):
        got = b.linear_mxfp4(*dev, bias=None if bi is None else bi.cuda(), activation=act,
                             residual=None if re is None else re.cuda(), out_dtype=DT[dt])
        assert got.dtype == DT[dt] and got.shape == (M, N)
        check(got, args, act, bi, re)


def test_scales_over_their_range(b):
    """Scales from 2^-60 to 2^60 a side, and the ends where one product is the sum."""
    g = np.random.default_rng(3)
    for M, N in ((4, 48), (64, 48), (400, 300)):
        c, _, w, _ = exact(M, N, 256, 5)
        cs, ws = (torch.from_numpy(g.integers(67, 188, (n, 8), dtype=np.uint8)) for n in (M, N))
        check(b.linear_mxfp4(*(t.cuda() for t in (c, cs, w, ws)), out_dtype=torch.float32), (c, cs, w, ws))
        c[:, 1:], w[:, 1:] = 0, 0
        for a, v in ((0, 250), (254, 0), (1, 250), (127, 127), (127, 5)):
            cs[:], ws[:] = 127, 127
            cs[:, 0], ws[:, 0] = a, v
            check(b.linear_mxfp4(*(t.cuda() for t in (c, cs, w, ws)), out_dtype=torch.float32), (c, cs, w, ws))


@pytest.mark.parametrize("M", [3, 40, 500])
def test_layouts(b, M):
    """Strided residual and output, leading dims, in place, nothing written beside."""
    N, K = 132, 384
    args, bias, residual = rough(M, N, K, M, torch.float16)
    dev = [t.cuda() for t in args]
    want = b.linear_mxfp4(*dev, bias=bias.cuda(), residual=residual.cuda())
    check(want, args, None, bias, residual)
    wide = torch.full((M, N + 9), 3.0, dtype=torch.float16, device="cuda")
    wide[:, 5:5 + N] = residual.cuda()
    view = wide[:, 5:5 + N]
    got = b.linear_mxfp4(*dev, bias=bias.cuda(), residual=view, out=view)
    assert got.data_ptr() == view.data_ptr() and torch.equal(got, want)
    assert (wide[:, :5] == 3).all() and (wide[:, 5 + N:] == 3).all()
    if M % 4 == 0:
        lead = b.linear_mxfp4(dev[0].view(4, M // 4, -1), dev[1].view(4, M // 4, -1), dev[2], dev[3], bias=bias.cuda(),
                              residual=residual.cuda().view(4, M // 4, N))
        assert torch.equal(lead.view(M, N), want)


@pytest.mark.parametrize("M,K", [(3, 1024), (16, 352), (60, 1024), (40, 8192), (300, 512), (500, 96)])
def test_scales_at_any_address(b, M, K):
    args = exact(M, 200, K, M)
    want = b.linear_mxfp4(*(t.cuda() for t in args), out_dtype=torch.float32)
    for off in (1, 2, 7):
        dev = [t.cuda() for t in args]
        for i in (1, 3):
            flat = torch.zeros(args[i].numel() + 16, dtype=torch.uint8, device="cuda")
            flat[off: off + args[i].numel()] = dev[i].view(-1)
            dev[i] = flat[off: off + args[i].numel()].view(args[i].shape)
        assert dev[1].data_ptr() % 4 == off % 4
        assert torch.equal(b.linear_mxfp4(*dev, out_dtype=torch.float32), want)


@pytest.mark.parametrize("M,N,K", [(8, 512, 8192), (8, 64, 16384), (40, 256, 8192), (300, 700, 1024)])
def test_captured_and_on_another_stream(b, M, N, K):
    args, bias, _ = rough(M, N, K, 1, torch.bfloat16)
    dev, bias = [t.cuda() for t in args], bias.cuda()
    call = lambda: b.linear_mxfp4(*dev, bias=bias, activation="silu", out_dtype=torch.bfloat16)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = call()
    side.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(3):
        dev[0].add_(17)                         # other codes, any byte is one
        graph.replay()
        eager = call()
        torch.cuda.synchronize()
        assert torch.equal(got, eager)


def test_binding_refusals(b):
    c, s, w, ws = (t.cuda() for t in exact(4, 8, 64, 0))
    bad = [(dict(codes=c.float()), TypeError), (dict(scales=s.cpu()), TypeError), (dict(scales=s[:, :1]), ValueError),
           (dict(codes=c.t()), ValueError), (dict(w_codes=w[:, :16].contiguous(), w_scales=ws[:, :1].contiguous()), ValueError),
           (dict(w_codes=w[0], w_scales=ws[0]), ValueError), (dict(activation="tanh"), ValueError),
           (dict(bias=torch.zeros(8).cuda()), TypeError), (dict(bias=torch.zeros(7, dtype=torch.float16).cuda()), ValueError),
           (dict(residual=torch.zeros(4, 9, dtype=torch.float16).cuda()), ValueError), (dict(out_dtype=torch.int8), TypeError),
           (dict(out=torch.zeros(4, 8).cuda()), ValueError)]
    for kw, err in bad:
        with pytest.raises(err):
            b.linear_mxfp4(**{**dict(codes=c, scales=s, w_codes=w, w_scales=ws), **kw})
    for x, err in ((torch.randn(4, 33).cuda(), ValueError), (torch.randn(4, 32), TypeError),
                   (torch.randn(4, 32).double().cuda(), TypeError), (torch.randn(0, 32).cuda(), ValueError)):
        with pytest.raises(err):
            b.quantize_mxfp4(x)
    with pytest.raises(TypeError):
        b.dequantize_mxfp4(c, s, out_dtype=torch.float64)
