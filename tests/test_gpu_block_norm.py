"""The norms before and after a block, its gate, scale and residual against the
formulas in 64 bits (GPU).

Tolerances, u = 2^-24 the binary32 half step, on top of those of the single
norm (32 u for a normed value before its rounding, 34 u for a row_scale):
v = u * g * scale carries 32 u (norm), 6 u (sigmoid: exp 4 u, the sum and the
quotient u each), 2 u (two products): 40 u |v|.  h adds u |h|.  The second
norm's root mean square moves by at most 40 u |v|_2 / |h|_2 + u, relatively.
Values below the smallest normal number lose up to 2^-149 a step more."""
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


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def gpu(t):
    return None if t is None else t.cuda()


def make(M, H, dt, seed, post=True, gate="row", pre=True, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    spread = torch.exp(0.7 * torch.randn(H, generator=g))
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=(scale * rnd(M, H) * spread).to(dt), residual=(3 * scale * rnd(M, H) * spread).to(dt),
                post_weight=(0.5 + 0.2 * rnd(H)).to(dt) if post else None,
                pre_weight=(1 + 0.3 * rnd(H)).to(dt) if pre else None,
                gate=None if gate is None else (2 * rnd(*((H,) if gate == "channel" else (M, H)))).to(dt))


def errors(s, act, scale, eps):
    """(h, its error, its rms's relative error) in 64 bits."""
    h, v = rows.block64(f64(s["x"]), f64(s["residual"]), f64(s["post_weight"]), f64(s["gate"]), act, scale, eps)
    e = 40 * U * np.abs(v) + U * np.abs(h) + 2.0 ** -147
    norm = np.sqrt((h * h).sum(axis=1, keepdims=True) + eps * h.shape[1])
    d = (40 * U * np.sqrt((v * v).sum(axis=1, keepdims=True))) / np.maximum(norm, 1e-300) + U
    return h, e, d


def close(got, s, act=None, scale=1.0, eps=1e-6):
    normed, total = got
    h, e, d = errors(s, act, scale, eps)
    half = torch.finfo(total.dtype).eps / 2
    off = np.abs(f64(total) - h)
    assert np.all(off <= e + (np.abs(h) + e) * half + SMALLEST[total.dtype] / 2), float((off - e).max())
    if s["pre_weight"] is None:
        assert normed is None
        return
    w = f64(s["pre_weight"])
    rstd = rows.rstd64(h, eps)
    want = h * rstd * w
    half = torch.finfo(normed.dtype).eps / 2
    e = np.abs(want) * (32 * U + d) + np.abs(w) * rstd * e
    off = np.abs(f64(normed) - want)
    tol = e + (np.abs(want) + e) * half + SMALLEST[normed.dtype] / 2
    assert np.all(off <= tol), float((off / tol).max())


def close8(got, s, c, act=None, scale=1.0, eps=1e-6):
    codes, row_scales, total = got
    h, e, d = errors(s, act, scale, eps)
    f = f64(s["pre_weight"]) * (1.0 if c is None else f64(c))
    t, et = h * f, np.abs(f) * e + 3 * U * np.abs(h * f)
    peak = np.abs(t).max(axis=1, keepdims=True)
    ep = et.max(axis=1, keepdims=True)
    assert np.all(np.abs(f64(codes) - t * 127 / peak) <= 0.5 + 127 * (et / peak + ep / peak + 4 * U))
    want = (peak / 127 * rows.rstd64(h, eps))[:, 0]
    assert np.all(np.abs(f64(row_scales) - want) <= want * (34 * U + d[:, 0] + (ep / peak)[:, 0]))
    half = torch.finfo(total.dtype).eps / 2
    assert np.all(np.abs(f64(total) - h) <= e + (np.abs(h) + e) * half + SMALLEST[total.dtype] / 2)


SHAPES = [(1, 1), (1, 7), (3, 8), (2, 9), (5, 31), (1, 5120), (16, 5120), (17, 512), (4, 8192), (3, 8185), (2, 4097),
          (1300, 257), (2500, 96), (1100, 8192)]
FORMS = [(True, "row", True, "sigmoid", 1.0), (True, "channel", True, None, 0.25), (False, "row", True, None, 1.5),
         (False, None, True, None, -0.75), (True, None, False, None, 1.0), (False, "channel", False, "sigmoid", 0.5)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,H", SHAPES)
def test_block_norm(b, M, H, dt):
    for i, (post, gate, pre, act, scale) in enumerate(FORMS):
        s = make(M, H, DT[dt], 7 * M + H + i, post, gate, pre)
        odt = list(DT.values())[i % 3]
        got = b.rms_norm_block(gpu(s["x"]), gpu(s["residual"]), gpu(s["post_weight"]), gpu(s["pre_weight"]),
                               gate=gpu(s["gate"]), gate_activation=act, scale=scale, out_dtype=odt)
        assert got[1].dtype == DT[dt] and (not pre or got[0].dtype == odt)
        close(got, s, act, scale)
        if pre:
            c = torch.exp(-4 + 0.5 * torch.randn(H)).to(torch.float16) if i % 2 else None
            close8(b.rms_norm_block_int8(gpu(s["x"]), gpu(s["residual"]), gpu(s["post_weight"]), gpu(s["pre_weight"]),
                                         gate=gpu(s["gate"]), gate_activation=act, scale=scale,
                                         channel_scales=gpu(c)), s, c, act, scale)


@pytest.mark.parametrize("dt", list(DT))
def test_plain_addition_gives_the_bits_of_the_single_norm(b, dt):
    s = {k: gpu(v) for k, v in make(33, 5121, DT[dt], 5, post=False, gate=None).items()}
    normed, total = b.rms_norm_block(s["x"], s["residual"], None, s["pre_weight"])
    want = b.rms_norm(s["x"], s["pre_weight"], s["residual"])
    assert torch.equal(normed, want[0]) and torch.equal(total, want[1])
    got = b.rms_norm_block_int8(s["x"], s["residual"], None, s["pre_weight"])
    for a, w in zip(got, b.rms_norm_int8(s["x"], s["pre_weight"], s["residual"])):
        assert torch.equal(a, w)


def test_rows_alone_give_the_bits_of_the_batch(b):
    s = {k: gpu(v) for k, v in make(700, 1000, torch.bfloat16, 6).items()}
    whole = b.rms_norm_block(s["x"], s["residual"], s["post_weight"], s["pre_weight"], gate=s["gate"])
    for m in (0, 311, 699):
        one = b.rms_norm_block(s["x"][m:m + 1], s["residual"][m:m + 1], s["post_weight"], s["pre_weight"],
                               gate=s["gate"][m:m + 1])
        assert torch.equal(one[0][0], whole[0][m]) and torch.equal(one[1][0], whole[1][m])


@pytest.mark.parametrize("dt", list(DT))
def test_strided_rows_and_leading_dims(b, dt):
    M, H = 9, 333
    s = make(M, H, DT[dt], 8)
    wide = {k: torch.full((M, H + 5 + i), 7.0, dtype=DT[dt]).cuda() for i, k in enumerate(("x", "residual", "gate"))}
    for k, v in wide.items():
        v[:, 1:H + 1] = s[k].cuda()
    views = {k: v[:, 1:H + 1] for k, v in wide.items()}
    post, pre = gpu(s["post_weight"]), gpu(s["pre_weight"])
    got = b.rms_norm_block(views["x"], views["residual"], post, pre, gate=views["gate"], out_dtype=torch.float32)
    close(got, s)
    d3 = lambda t: gpu(t).view(3, 3, H)  # noqa: E731
    again = b.rms_norm_block(d3(s["x"]), d3(s["residual"]), post, pre, gate=d3(s["gate"]), out_dtype=torch.float32)
    assert again[0].shape == (3, 3, H) and torch.equal(again[0].view(M, H), got[0])
    assert torch.equal(again[1].view(M, H), got[1])
    for k, v in wide.items():                   # nothing around the views was written
        assert torch.all(v[:, 0] == 7) and torch.all(v[:, H + 1:] == 7)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("e", [-60, -45, 45, 60])
def test_rows_whose_squares_leave_binary32(b, dt, e):
    """eps 0 and rows of 2^e times the usual size: both norms stay what the formulas say."""
    for gate in (None, "channel"):
        s = make(5, 777, DT[dt], e + 100, gate=gate, scale=2.0 ** e)
        s["x"][1] *= 2.0 ** 10                  # rows of other sizes beside them
        s["residual"][2] *= 2.0 ** -8
        s["x"][3], s["residual"][3] = s["x"][3] * 2.0 ** -e, s["residual"][3] * 2.0 ** -e
        dev = {k: gpu(v) for k, v in s.items()}
        close(b.rms_norm_block(dev["x"], dev["residual"], dev["post_weight"], dev["pre_weight"], gate=dev["gate"],
                               eps=0.0, out_dtype=torch.float32), s, eps=0.0)
        close8(b.rms_norm_block_int8(dev["x"], dev["residual"], dev["post_weight"], dev["pre_weight"],
                                     gate=dev["gate"], eps=0.0), s, None, eps=0.0)


def test_gates_at_their_ends(b):
    """Sigmoids of gates over all of binary32; one below 2^-126, the smallest normal number, may count as 0."""
    z = torch.cat([torch.linspace(-110, 110, 4001), torch.tensor([0.0, -0.0, 1e-38, -1e-38, 1e30, -1e30, 3e38, -3e38,
                                                                  float("inf"), -float("inf"), 87.5, -87.5, 1e-4, -1e-4])])
    H = len(z)
    x, r = torch.full((2, H), 3.0), torch.zeros(2, H)
    total = b.rms_norm_block(x.cuda(), r.cuda(), gate=z.cuda(), gate_activation="sigmoid")[1]
    want = 3.0 / (1.0 + np.exp(-f64(z)))
    assert np.all(np.abs(f64(total) - want) <= 40 * U * want + U * want + 3.0 * 2.0 ** -126)
    z[7] = float("nan")
    total = b.rms_norm_block(x.cuda(), r.cuda(), gate=z.cuda(), gate_activation="sigmoid")[1].cpu()
    assert total[:, 7].isnan().all() and total.isnan().sum() == 2


def test_bad_values_stay_in_their_rows(b):
    s = make(6, 600, torch.float32, 9)
    clean = {k: gpu(v) for k, v in s.items()}
    want = b.rms_norm_block(*(clean[k] for k in ("x", "residual", "post_weight", "pre_weight")), gate=clean["gate"])
    s["x"][1, 3], s["residual"][2, 5], s["gate"][3, 7], s["x"][4, 9] = np.nan, np.inf, -np.inf, np.inf
    bad = {k: gpu(v) for k, v in s.items()}
    got = b.rms_norm_block(*(bad[k] for k in ("x", "residual", "post_weight", "pre_weight")), gate=bad["gate"])
    for m in (0, 5):
        assert torch.equal(got[0][m], want[0][m]) and torch.equal(got[1][m], want[1][m])
    assert got[0][1].isnan().all() and got[1][1].isnan().all()
    assert got[1][2, 5] == np.inf and got[0][2, 5].isnan() and (got[0][2].nan_to_num(0) == 0).all()
    assert got[1][3, 7].isinf() and got[1][4, 9].isnan()
    codes, row_scales, _ = b.rms_norm_block_int8(*(bad[k] for k in ("x", "residual", "post_weight", "pre_weight")),
                                                 gate=bad["gate"])
    for m in (1, 2, 3, 4):
        assert (codes[m] == 0).all() and not row_scales[m].isfinite()


def test_captured_and_on_another_stream(b):
    s = {k: gpu(v) for k, v in make(40, 2048, torch.float16, 10).items()}
    call = lambda: b.rms_norm_block(s["x"], s["residual"], s["post_weight"], s["pre_weight"],  # noqa: E731
                                    gate=s["gate"], gate_activation="sigmoid")
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = call()
    side.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(3):
        s["x"].mul_(-1.0)
        graph.replay()
        eager = call()
        torch.cuda.synchronize()
        assert torch.equal(got[0], eager[0]) and torch.equal(got[1], eager[1])


def test_sum_written_over_its_inputs(b):
    """The C entry's sum_out may be x, the residual or a gate of rows."""
    L = b.load_library()
    s = {k: gpu(v) for k, v in make(21, 640, torch.bfloat16, 11).items()}
    want = b.rms_norm_block(s["x"], s["residual"], s["post_weight"], s["pre_weight"], gate=s["gate"])
    for over in ("x", "residual", "gate"):
        c = {k: v.clone() for k, v in s.items()}
        out = torch.empty(21, 640, dtype=torch.float16, device="cuda")
        st = L.rms_norm_block_rows(c["x"].data_ptr(), 640, c["residual"].data_ptr(), 640, c["gate"].data_ptr(), 640,
                                   0, 1, c["post_weight"].data_ptr(), c["pre_weight"].data_ptr(), 1, 1.0, 21, 640,
                                   1e-6, c[over].data_ptr(), out.data_ptr(), 0, b._stream_ptr(out.device))
        assert st == 0
        assert torch.equal(out, want[0]) and torch.equal(c[over], want[1])


def test_binding_refusals(b):
    s = {k: gpu(v) for k, v in make(4, 64, torch.float16, 12).items()}
    ok = dict(x=s["x"], residual=s["residual"], post_weight=s["post_weight"], pre_weight=s["pre_weight"])
    bad = [(dict(residual=s["residual"].float()), ValueError), (dict(residual=s["residual"][:3]), ValueError),
           (dict(post_weight=s["post_weight"][:63]), ValueError), (dict(post_weight=s["post_weight"].float()), TypeError),
           (dict(pre_weight=s["pre_weight"].cpu()), TypeError), (dict(gate=s["gate"].float()), TypeError),
           (dict(gate=s["gate"][:, :32]), ValueError), (dict(gate=s["gate"], gate_activation="tanh"), ValueError),
           (dict(gate_activation="sigmoid"), ValueError), (dict(out_dtype=torch.int8), TypeError),
           (dict(x=s["x"].t()), ValueError), (dict(scale=float("nan")), RuntimeError), (dict(eps=-1.0), RuntimeError)]
    for kw, err in bad:
        with pytest.raises(err):
            b.rms_norm_block(**{**ok, **kw})
    with pytest.raises(ValueError):
        b.rms_norm_block_int8(s["x"], s["residual"], None, None)
