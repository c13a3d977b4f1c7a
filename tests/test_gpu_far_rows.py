"""Rows, codes and outputs behind 2^32 bytes or elements (GPU): block norms,
rows in 4-bit floating point and their products."""
import pytest
import torch

from oracle import mxfp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def test_block_norm_rows_far_apart(b):
    far = (1 << 32) + 64
    g = torch.Generator().manual_seed(1)
    x, r, gate = (torch.randn(2, 264, generator=g).half().cuda() for _ in range(3))
    w = torch.rand(264, generator=g).half().cuda()
    buf = torch.empty(far + 3 * 320, dtype=torch.float16, device="cuda")
    views = [torch.as_strided(buf, (2, 264), (far, 1), 320 * i) for i in range(3)]
    for v, t in zip(views, (x, r, gate)):
        v.copy_(t)
    want = b.rms_norm_block(x, r, w, w, gate=gate)
    got = b.rms_norm_block(views[0], views[1], w, w, gate=views[2])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want8 = b.rms_norm_block_int8(x, r, w, w, gate=gate)
    for a, e in zip(b.rms_norm_block_int8(views[0], views[1], w, w, gate=views[2]), want8):
        assert torch.equal(a, e)


def test_quantize_many_rows(b):
    """2^32 + 2^15 channels: contiguous, and the last rows by themselves."""
    M, H = (1 << 19) + 4, 8192
    x = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    x.random_(-100, 100)
    codes, scales = b.quantize_mxfp4(x)
    back = b.dequantize_mxfp4(codes, scales, out_dtype=torch.bfloat16)
    for at in (0, 1 << 18, (1 << 19) - 2, M - 3):
        part = x[at: at + 3].contiguous()
        c, s = b.quantize_mxfp4(part)
        assert torch.equal(c, codes[at: at + 3]) and torch.equal(s, scales[at: at + 3])
        assert torch.equal(b.dequantize_mxfp4(c, s, out_dtype=torch.bfloat16), back[at: at + 3])


def test_quantize_more_chunks_than_a_grid_has_threads(b):
    """2^35 + 2^18 channels, 8 of them a thread."""
    M, H = (1 << 19) + 4, 65536
    x = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    x.random_(-100, 100)
    codes, scales = b.quantize_mxfp4(x)
    at = [0, (1 << 18) - 1, 1 << 18, (1 << 19) - 1, 1 << 19, M - 1]
    want = [b.quantize_mxfp4(x[i: i + 1].contiguous()) for i in at]
    del x
    back = b.dequantize_mxfp4(codes, scales, out_dtype=torch.bfloat16)
    for i, (c, s) in zip(at, want):
        assert torch.equal(c[0], codes[i]) and torch.equal(s[0], scales[i])
        assert torch.equal(b.dequantize_mxfp4(c, s, out_dtype=torch.bfloat16)[0], back[i])


def operands(n, K):
    """Codes whose products' sums are quarters below 2^24, made on the device."""
    c = torch.empty(n, K // 2, dtype=torch.uint8, device="cuda")
    c.random_(0, 256)
    return c, torch.full((n, K // 32), 127, dtype=torch.uint8, device="cuda")


def values(c, s):
    return torch.from_numpy(mxfp4.values(c.cpu().numpy(), s.cpu().numpy()))


@pytest.mark.parametrize("M,N,K", [((1 << 20) - 3, 40, 8224), (3, (1 << 20) + 40, 8224), (70, (1 << 20) + 40, 8224),
                                   (200, (1 << 20) + 40, 8224), (1100, 4 << 20, 32)])
def test_products_far_out(b, M, N, K):
    """Codes behind 2^32 bytes on either side, and outputs behind 2^32 elements."""
    x, xs = operands(M, K)
    w, ws = operands(N, K)
    got = b.linear_mxfp4(x, xs, w, ws, out_dtype=torch.float32)
    m = sorted({0, M // 2, max(0, M - 2), M - 1})
    n = sorted({0, 1, N // 2, N - 17, N - 2, N - 1})
    want = values(x[m], xs[m]) @ values(w[n], ws[n]).T.contiguous()
    assert torch.equal(got[m][:, n].double().cpu(), want)
