"""The largest numbers of rows, columns and tokens that the entry points take
(GPU): exact sums and selections, on every row or on rows from all over."""
import numpy as np
import pytest
import torch

from oracle import logit_rules as lr
from tests.test_gpu_logit_rules import dev, device_rules, make, same
from tests.test_gpu_logit_rules_chunks import check, uniforms

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def unpack(w):
    p = w.int()
    q = torch.stack((p & 15, p >> 4), dim=2).view(p.shape[0], -1)
    return torch.where(q > 7, q - 16, q).double()


@pytest.mark.parametrize("M,N,K", [(1 << 20, 40, 64), ((1 << 20) - 3, 129, 32), (2, 1 << 24, 32), (20, 1 << 24, 32),
                                   (16, (1 << 24) - 5, 32), (100, 3, 65536), (5, 70, 65536)])
def test_linear(b, M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M ^ N)
    w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    codes = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    got = b.linear_int4(codes, torch.ones(M, device="cuda"), w, out_dtype=torch.float32)
    # sums below 2^26 at K = 65536: one rounding to binary32
    if M > 4096:
        want = codes.double() @ unpack(w).t().contiguous()
        assert torch.equal(got, want.float())
    else:
        step = 1 << 20
        for lo in range(0, N, step):
            want = codes.double() @ unpack(w[lo: lo + step]).t().contiguous()
            assert torch.equal(got[:, lo: lo + step], want.float())


def test_norm_of_a_million_rows(b):
    M, H = (1 << 20) + 7, 96
    x = torch.randn(M, H, device="cuda").half()
    w = torch.rand(H, device="cuda").half()
    y, total = b.rms_norm(x, w, x)
    h = 2 * x.float()
    want = h.double() * torch.rsqrt((h.double() ** 2).mean(1, keepdim=True) + 1e-6) * w.double()
    u = 2.0 ** -24
    off = (y.double() - want).abs()
    assert bool((off <= want.abs() * (2.0 ** -11 + 33 * u) + 2.0 ** -25).all())
    assert torch.equal(total, h.half())
    q, s = b.quantize_rows(x)
    peak = x.float().abs().amax(1, keepdim=True)
    assert torch.equal(q, torch.round(x.float() * (torch.full_like(peak, 127.0) / peak)).to(torch.int8))


@pytest.mark.parametrize("R,T,V", [(4096, 1, 500), (256, 16, 1500), (1365, 3, 2000)])
def test_rules_on_4096_rows(b, R, T, V):
    logits, rules, drafts = make(R, T, V, 3, history=20, bias=3)
    x, r, d = dev(logits), device_rules(b, rules), dev(drafts) if T > 1 else None
    want = lr.ruled(logits, rules, drafts, R, T)
    same(b.apply_logit_rules(x, r, d, R=R), want)
    ruled = torch.from_numpy(want).cuda()
    for k in (0, 16):
        check(b.verify_logits(x, r, d, R=R, top_k=k, want_lse=True), ruled, d, None, None, R, T, k, 1.0)
        if T > 1:
            dp, un = uniforms(R, T, 1)
            check(b.verify_logits(x, r, d, dp, un, R=R, top_k=k), ruled, d, dp, un, R, T, k, 1.0)


@pytest.mark.parametrize("R,T,V,H", [(4096, 1, 300, 32), (256, 16, 700, 64)])
def test_ruled_verification_of_4096_rows(b, R, T, V, H):
    from int4_output_head_amd import synth
    i = synth.int_exact_inputs(R * T, V, H, seed=V)
    h = torch.from_numpy(i["hidden"]).view(torch.float16).cuda()
    w, s = torch.from_numpy(i["packed"]).cuda(), torch.from_numpy(i["scales"]).view(torch.float16).cuda()
    _, rules, drafts = make(R, T, V, 4, history=20, bias=3)
    r, d = device_rules(b, rules), dev(drafts) if T > 1 else None
    logits = b.verify_batch(h, w, s, d, R=R, logits=True)[3]
    ruled = torch.from_numpy(lr.ruled(logits.cpu().numpy(), rules, drafts, R, T)).cuda()
    for k in (0, 5):
        check(b.verify_ruled(h, w, s, r, d, R=R, top_k=k, want_lse=True), ruled, d, None, None, R, T, k, 1.0)


def test_rules_on_2_24_tokens(b):
    R, T, V = 1, 2, 1 << 24
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(T, V, generator=g, device="cuda")
    last = V - 1
    rules = dict(lr.NONE, history=np.array([0, last, last, 5], np.int32), history_offsets=np.array([0, 4]),
                 n_prompt=np.array([1], np.int32), presence=np.array([0.5], np.float32),
                 frequency=np.array([0.25], np.float32), bias_ids=np.array([last, 7, V], np.int32),
                 bias_values=np.array([30.0, 20.0, 99.0], np.float32), bias_offsets=np.array([0, 3]))
    words = np.full((2, V // 32), 0xFFFFFFFF, np.uint32)
    words[0, 0] &= ~np.uint32(1 << 3)
    words[1, -1] &= np.uint32(0x7FFFFFFF)              # the last token is refused in row 1
    rules["mask"] = words
    d = torch.tensor([[last]], dtype=torch.int32, device="cuda")
    want = x.clone()
    want[:, 5] -= 0.25
    want[:, 5] -= 0.5
    for t, count in ((0, 2.0), (1, 3.0)):
        want[t, last] = want[t, last] - 0.25 * count - 0.5 + 30.0
        want[t, 7] += 20.0
    want[0, 3] = -float("inf")
    want[1, last] = -float("inf")
    r = device_rules(b, rules)
    assert torch.equal(b.apply_logit_rules(x, r, d, R=R), want)
    for k in (0, 16):
        got = b.verify_logits(x, r, d, R=R, top_k=k, want_lse=True)
        assert got[1].tolist() == [last, 7] and got[5].tolist() == [1]
        check(got, want, d, None, None, R, T, k, 1.0)
