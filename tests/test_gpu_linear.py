"""The int4 linear layer against its formula in 64 bits (GPU).

Tolerances, u = 2^-24.  The integer sum is exact (below 2^24 at these sizes).
s = acc * row_scale * out_scale: 2 u |s|; + bias: u |y|; so d = 3 u |s| + u |y|
in front of the activation, whose slope is at most 1.13 (gelu), plus its own
8 u |y| (erf, exp, quotient, products: each a few units at most), plus u (|z| +
|residual|) for the last sum, then half a step of the output's type or half of
its smallest step."""
import numpy as np
import pytest
import torch

from int4_output_head_amd import synth
from oracle import rows

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SMALLEST = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133, torch.float32: 2.0 ** -149}


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def make(M, N, K, seed, dt=torch.float16, extreme=False):
    g = np.random.default_rng(seed)
    codes = g.integers(-128 if extreme else -127, 128, (M, K)).astype(np.int8)
    q = g.integers(-8 if extreme else -7, 8, (N, K)).astype(np.int8)
    if extreme:
        codes[:, :] = -128
        q[::2] = -8
    rs = np.exp(g.normal(-7, 0.4, M)).astype(np.float32)
    return dict(codes=torch.from_numpy(codes), row_scales=torch.from_numpy(rs),
                packed=torch.from_numpy(synth.pack_int4(q)),
                out_scales=torch.from_numpy(np.exp(g.normal(-1, 0.3, N)).astype(np.float32)),
                bias=torch.from_numpy(g.normal(0, 0.5, N).astype(np.float32)).to(dt),
                residual=torch.from_numpy(g.normal(0, 1, (M, N)).astype(np.float32)).to(dt))


def call(b, d, dt, act=None, out_scales=True, bias=True, residual=True, **kw):
    c = {k: v.cuda() for k, v in d.items()}
    return b.linear_int4(c["codes"], c["row_scales"], c["packed"], out_scales=c["out_scales"] if out_scales else None,
                         bias=c["bias"] if bias else None, activation=act, residual=c["residual"] if residual else None,
                         out_dtype=dt, **kw)


def check(got, d, act=None, out_scales=True, bias=True, residual=True):
    f = lambda k, use: d[k].double().numpy() if use else None  # noqa: E731
    z, y, s = rows.linear64(d["codes"].numpy(), d["row_scales"].double().numpy(), d["packed"].numpy(),
                            f("out_scales", out_scales), f("bias", bias), act, f("residual", residual))
    tol = 1.13 * (3 * U * np.abs(s) + U * np.abs(y)) + (8 * U * np.abs(y) if act in ("gelu", "silu") else 0)
    if residual:
        tol = tol + U * (np.abs(z) + np.abs(d["residual"].double().numpy()) + tol)
    tol = tol + torch.finfo(got.dtype).eps / 2 * (np.abs(z) + tol) + SMALLEST[got.dtype] / 2
    off = np.abs(got.cpu().double().numpy() - z)
    assert np.all(off <= tol), float((off / tol).max())


SHAPES = [(1, 1, 32), (1, 16, 64), (1, 5120, 5120), (3, 17, 96), (16, 512, 5120), (16, 100, 8192), (17, 333, 2048),
          (32, 64, 1024), (32, 1000, 8192), (1, 40, 8224), (20, 33, 20480), (33, 65, 160), (64, 128, 128), (50, 300, 4096),
          (65, 129, 352), (128, 256, 1024), (200, 127, 8192), (300, 513, 640), (257, 1030, 512), (1000, 100, 2080),
          (130, 3, 64), (2100, 2600, 32), (4096, 4097, 64)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(b, M, N, K):
    d = make(M, N, K, M + N + K)
    check(call(b, d, torch.float16, "silu"), d, "silu")


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("act", [None, "relu", "gelu", "silu"])
@pytest.mark.parametrize("M,N,K", [(5, 70, 256), (40, 70, 256), (150, 131, 4096), (260, 300, 96)])
def test_epilogue(b, M, N, K, act, dt):
    d = make(M, N, K, M + len(dt), DT[dt])
    for out_scales, bias, residual in ((True, True, True), (False, True, False), (True, False, False),
                                       (False, False, True), (False, False, False)):
        got = call(b, d, DT[dt], act, out_scales, bias, residual)
        assert got.dtype == DT[dt] and got.shape == (M, N)
        check(got, d, act, out_scales, bias, residual)


@pytest.mark.parametrize("M,N,K", [(2, 64, 8192), (40, 64, 8192), (300, 300, 8192), (4, 16, 65536), (70, 20, 65536)])
def test_largest_sums(b, M, N, K):
    """codes -128 against weights -8: the largest sum an int32 has to hold."""
    d = make(M, N, K, 1, extreme=True)
    got = call(b, d, torch.float32, None, False, False, False)
    acc = d["codes"].numpy().astype(np.int64) @ rows.unpack_int4(d["packed"].numpy()).T
    want = acc.astype(np.float64) * d["row_scales"].double().numpy()[:, None]
    assert acc.max() == 128 * 8 * K
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= 3 * U * np.abs(want))


def test_a_row_gives_the_same_bits_in_every_batch(b):
    d = make(600, 777, 5120, 3, torch.float32)
    whole = call(b, d, torch.float32, "gelu")
    for lo, hi in ((0, 1), (5, 21), (30, 62), (100, 150), (17, 217), (64, 464)):
        part = {k: v[lo:hi] if k in ("codes", "row_scales", "residual") else v for k, v in d.items()}
        assert torch.equal(call(b, part, torch.float32, "gelu"), whole[lo:hi]), (lo, hi)


@pytest.mark.parametrize("M,N,K", [(4, 37, 128), (48, 130, 128), (300, 300, 4096)])
def test_strides_and_rows_behind(b, M, N, K):
    d = make(M, N, K, 8)
    want = call(b, d, torch.float16)
    c = {k: v.cuda() for k, v in d.items()}
    codes = torch.zeros(M + 2, K + 48, dtype=torch.int8, device="cuda")
    codes[:M, 16: 16 + K] = c["codes"]
    res = torch.full((M + 3, N + 7), 9.0, dtype=torch.float16, device="cuda")
    res[:M, 5: 5 + N] = c["residual"]
    keep = res.clone()
    out = torch.full((M + 2, N + 3), 7.0, dtype=torch.float16, device="cuda")
    kw = dict(out_scales=c["out_scales"], bias=c["bias"])
    got = b.linear_int4(codes[:M, 16: 16 + K], c["row_scales"], c["packed"], residual=res[:M, 5: 5 + N],
                        out=out[:M, 1: 1 + N], **kw)
    assert torch.equal(got, want)
    assert torch.equal(res, keep)
    out[:M, 1: 1 + N] = 7.0
    assert torch.equal(out, torch.full_like(out, 7.0))
    # onto the residual itself
    b.linear_int4(codes[:M, 16: 16 + K], c["row_scales"], c["packed"], residual=res[:M, 5: 5 + N],
                  out=res[:M, 5: 5 + N], **kw)
    assert torch.equal(res[:M, 5: 5 + N], want)
    res[:M, 5: 5 + N] = keep[:M, 5: 5 + N]
    assert torch.equal(res, keep)


def test_non_finite_row_scales(b):
    for M in (3, 40):
        d = make(M, 50, 64, 4)
        d["row_scales"][1] = float("nan")
        d["row_scales"][2] = float("inf")
        d["codes"][2] = 0
        got = call(b, d, torch.float32, "relu", bias=False, residual=False).cpu()
        assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all()
        assert torch.isfinite(got[0]).all()


def test_streams_and_graphs(b):
    """Two graphs and the eager calls between their replays, with a split sum
    (a workspace) among them."""
    shapes = ((9, 64, 20480), (80, 100, 8192), (260, 300, 512))
    ds = [{k: v.cuda() for k, v in make(*s, 6).items()} for s in shapes]
    run = lambda: [b.linear_int4(d["codes"], d["row_scales"], d["packed"], bias=d["bias"]) for d in ds]  # noqa: E731
    run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    for k in range(3):
        for d in ds:
            d["codes"].copy_(torch.randint(-127, 128, d["codes"].shape, dtype=torch.int8))
        want = run()
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for u, v in zip(out, want):
                assert torch.equal(u, v)
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for s in side:
        with torch.cuda.stream(s):
            outs.append(run())
    torch.cuda.synchronize()
    for out in outs:
        for u, v in zip(out, want):
            assert torch.equal(u, v)


def test_refusals(b):
    d = {k: v.cuda() for k, v in make(4, 32, 64, 0).items()}
    c, s, w = d["codes"], d["row_scales"], d["packed"]
    for bad in (lambda: b.linear_int4(c, s[:3], w), lambda: b.linear_int4(c[:, :32], s, w),
                lambda: b.linear_int4(c, s, w, activation="tanh"), lambda: b.linear_int4(c, s, w, out_scales=s),
                lambda: b.linear_int4(c, s, w, bias=d["bias"][:5]), lambda: b.linear_int4(c, s, w, residual=d["residual"][:2]),
                lambda: b.linear_int4(c, s, w, out=torch.empty(4, 31, dtype=torch.float16, device="cuda")),
                lambda: b.linear_int4(c.t(), s, w)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: b.linear_int4(c.int(), s, w), lambda: b.linear_int4(c, s.double(), w),
                lambda: b.linear_int4(c, s, w, bias=d["bias"].float()), lambda: b.linear_int4(c, s, w.cpu()),
                lambda: b.linear_int4(c, s, w, out_dtype=torch.float64)):
        with pytest.raises(TypeError):
            bad()
    wide = torch.zeros(4, 72, dtype=torch.int8, device="cuda")
    with pytest.raises(RuntimeError):          # rows that are not 16-byte aligned
        b.linear_int4(wide[:, :64], s, w)
