"""Tokens drawn from logits against the definitions in 64 bits (GPU).

Tokens are equal to the oracle's unless a border lies within 2^-32 of the
whole mass of where it was asked for: masses of binary64 carry 2^-50, and each of
up to 2^18 tokens is rounded to a multiple of 2^-44 of the largest, 2^-45 * 2^18 at
most where all roundings go one way and 2^-36 as a sum of independent ones.
Probabilities: one rounding to binary32 beside those: 2^-24 + 2^-32, relatively,
and 2^-32 of a token's own unit where its mass is small."""
import math

import numpy as np
import pytest
import torch

from oracle import logit_rules as lr
from oracle import sampling

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEAR = 2.0 ** -32


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def gpu(t):
    return None if t is None else t.cuda()


def logits(M, V, dt, seed, spread=2.0):
    """A power law over some tokens, the rest far below."""
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(M, V, generator=g)
    n = max(1, min(V // 2, 300))
    at = torch.argsort(torch.rand(M, V, generator=g), dim=1)[:, :n] if V < 20000 else \
        torch.arange(n) * (V // n) + torch.randint(0, V // n, (M, n), generator=g)
    rank = 1 + torch.argsort(torch.rand(M, n, generator=g), dim=1).float()
    x.scatter_(1, at, 16.0 - 1.3 * torch.log(rank) + 0.5 * torch.randn(M, n, generator=g))
    return x.to(dt)


def allowed(row, setting, u, d):
    """Tokens that a border's nearness leaves open, and the draft's probability."""
    t, k, p, m = setting
    open_, shares = set(), []
    for e in ({0.0} if p >= 1 or p <= 0 else {-NEAR, 0.0, NEAR}):
        tokens = sampling.kept(row, t, k, p * (1 + e) if p < 1 else p, m) if e else sampling.kept(row, t, k, p, m)
        shares.append(0.0 if d is None else sampling.p_draft(row, tokens, t, d))
        lo, hi = (sampling.draw(row, tokens, t, u * (1 + s) + s if u == u else 0.0, d)[0] for s in (-NEAR, NEAR))
        left = tokens[tokens != d] if d is not None else tokens
        open_ |= {int(v) for v in left[(left >= lo) & (left <= hi)]} or {-1}
    return open_, shares


def check(got, rows, settings, uniforms, drafts=None, accept=None, R=None, T=1):
    """rows: the ruled logits as numpy; settings: a (temperature, top_k, top_p,
    min_p) per request."""
    ids, probs, pdr, nacc = (None if t is None else t.cpu().numpy() for t in got)
    M = len(rows)
    R = R or M // T
    u = uniforms.reshape(-1).tolist()
    for r in range(M):
        i, t = divmod(r, T)
        d = int(drafts[i, t]) if accept is not None and t < T - 1 else None
        open_, shares = allowed(rows[r], settings[i], u[r], d)
        assert int(ids[r]) in open_, (r, int(ids[r]), sorted(open_)[:5], settings[i], u[r])
        tokens = sampling.kept(rows[r], *settings[i])
        left = tokens[tokens != d] if d is not None else tokens
        if ids[r] < 0:
            assert probs[r] == 0
        else:
            temp = settings[i][0]
            ms = sampling.masses(rows[r][left], temp) if 0 < temp < math.inf else np.ones(len(left))
            want = ms[left == ids[r]][0] / ms.sum() if ids[r] in left else float(probs[r])
            assert abs(probs[r] - want) <= want * (2.0 ** -24 + NEAR) + 2.0 ** -60, (r, probs[r], want)
        if d is not None:
            assert min(abs(pdr[i, t] - s) for s in shares) <= pdr[i, t] * (2.0 ** -24 + NEAR) + 2.0 ** -60
    if accept is not None:
        for i in range(R):
            n = next((t for t in range(T - 1) if not accept[i, t] < pdr[i, t]), T - 1)
            assert nacc[i] == n


SETTINGS = [(1.0, 0, 1.0, 0.0), (0.5, 0, 1.0, 0.0), (2.0, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (1.0, 1, 1.0, 0.0),
            (0.8, 5, 1.0, 0.0), (1.0, 50, 0.95, 0.0), (1.0, 64, 1.0, 0.05), (1.3, 65, 0.9, 0.0), (1.0, 1000, 1.0, 0.0),
            (1.0, 0, 0.1, 0.0), (0.7, 0, 0.5, 0.0), (1.0, 0, 0.9, 0.0), (1.5, 0, 0.999, 0.0), (1.0, 0, 0.0, 0.0),
            (1.0, 0, 1.0, 0.01), (2.0, 0, 1.0, 0.5), (1.0, 0, 1.0, 1.0), (1.0, 0, 0.95, 0.02), (0.9, 40, 0.8, 0.1),
            (0.01, 0, 1.0, 0.0), (100.0, 0, 1.0, 0.0), (100.0, 30, 0.5, 0.0)]
SIZES = [(1, 1), (1, 2), (3, 7), (40, 64), (5, 1000), (3, 1024), (2, 1025), (7, 8191), (2, 20001), (300, 701)]


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("M,V", SIZES)
def test_settings(b, M, V, dt):
    x = logits(M, V, DT[dt], M + V)
    g = torch.Generator().manual_seed(V)
    for s in SETTINGS:
        u = torch.rand(M, generator=g)
        got = b.sample_logits(x.cuda(), u.cuda(), R=M, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        assert got[2] is None and got[3] is None
        if M <= 40:
            check(got, x.double().numpy(), [s] * M, u)
        else:
            keep = [0, 1, 7, 150, 299]
            check([None if t is None else t[keep] for t in got], x[keep].double().numpy(), [s] * 5, u[keep])


@pytest.mark.parametrize("V", [151936, 300000])
def test_long_rows(b, V):
    x = logits(3, V, torch.float32, V)
    u = torch.tensor([0.0, 0.37, 1 - 2.0 ** -24])
    for s in SETTINGS:
        got = b.sample_logits(x.cuda(), u.cuda(), R=3, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        check(got, x.double().numpy(), [s] * 3, u)


def test_settings_of_each_request(b):
    """Device settings, out-of-range ones among them, equal to the scalars' results bit for bit."""
    odd = [(-1.0, 3, 0.5, 0.1), (math.nan, 3, 0.5, 0.1), (math.inf, 3, 0.5, 0.1), (1.0, -4, math.nan, math.nan),
           (1.0, 5000, 1.5, -0.5), (1.0, 0, -0.5, 0.0), (1.0, 0, 1.0, 3.0)]
    plain = [(0.0, 0, 1.0, 0.0)] * 3 + [(1.0, 0, 1.0, 0.0)] * 2 + [(1.0, 0, 0.0, 0.0), (1.0, 0, 1.0, 1.0)]
    every, means = SETTINGS + odd, SETTINGS + plain
    R, T, V = len(every), 2, 3001
    x = logits(R * T, V, torch.float32, 1).cuda()
    u = torch.rand(R * T).cuda()
    d = torch.randint(0, V, (R, 1), dtype=torch.int32).cuda()
    t, k, p, m = (torch.tensor([s[i] for s in every], dtype=torch.int32 if i == 1 else torch.float32).cuda()
                  for i in range(4))
    got = b.sample_logits(x, u, None, d, R=R, temperature=t, top_k=k, top_p=p, min_p=m)
    for i, s in enumerate(means):
        one = b.sample_logits(x[2 * i:2 * i + 2], u[2 * i:2 * i + 2], None, d[i:i + 1], R=1, temperature=s[0], top_k=s[1],
                              top_p=s[2], min_p=s[3])
        assert torch.equal(got[0][2 * i:2 * i + 2], one[0]) and torch.equal(got[1][2 * i:2 * i + 2], one[1])
    check(got, x.cpu().double().numpy(), means, u.cpu(), T=T)


@pytest.mark.parametrize("V", [1000, 8192, 9000, 30000])
def test_equal_logits(b, V):
    """Ties go to the lower token; rows with more candidates than LDS holds."""
    x = torch.full((5, V), 3.25)
    x[1, V // 2:] = 3.0
    x[2, ::3] = 3.5
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24])
    for s in ((1.0, 0, 1.0, 0.0), (1.0, 10, 1.0, 0.0), (1.0, V - 1, 1.0, 0.0), (1.0, 0, 0.5, 0.0), (0.0, 0, 1.0, 0.0),
              (1.0, 700, 0.3, 0.0), (1.0, 0, 1.0, 0.8), (1.0, 0, 0.9999, 0.0)):
        got = b.sample_logits(x.cuda(), u.cuda(), R=5, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        check(got, x.double().numpy(), [s] * 5, u)
    # by hand: uniform over the first k
    got = b.sample_logits(x[:1].cuda(), torch.tensor([0.95]).cuda(), R=1, top_k=10)
    assert got[0].item() == 9 and abs(got[1].item() - 0.1) < 1e-8


def test_uniform_numbers_at_their_ends(b):
    x = logits(1, 777, torch.float32, 3).expand(7, 777).contiguous()
    u = torch.tensor([0.0, -1.0, float("nan"), 1.0, 2.0, 1 - 2.0 ** -24, float("inf")])
    for s in ((1.0, 0, 1.0, 0.0), (1.0, 9, 1.0, 0.0)):
        ids = b.sample_logits(x.cuda(), u.cuda(), R=7, temperature=s[0], top_k=s[1])[0].tolist()
        tokens = sampling.kept(x[0].double().numpy(), *s)
        assert ids[0] == ids[1] == ids[2] == tokens[0]
        assert ids[3] == ids[4] == ids[6] == tokens[-1]


def test_infinities_and_nan(b):
    V = 2100
    x = logits(8, V, torch.float32, 4)
    x[0, :] = -math.inf
    x[1, :] = math.nan
    x[2, 5:] = -math.inf
    x[3, [7, 1900]] = math.inf
    x[4, ::2] = math.nan
    x[5, 3] = -math.inf
    x[6, 100] = math.nan
    x[6, :100] = torch.finfo(torch.float32).min
    x[7, :] = torch.finfo(torch.float32).max
    u = torch.linspace(0, 0.999, 8)
    for s in SETTINGS:
        got = b.sample_logits(x.cuda(), u.cuda(), R=8, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        assert got[0][:2].tolist() == [-1, -1] and got[1][:2].tolist() == [0, 0]
        check(got, x.double().numpy(), [s] * 8, u)


def speculative(R, T, V, seed, dt=torch.float32):
    x = logits(R * T, V, dt, seed)
    g = torch.Generator().manual_seed(seed)
    best = x.float().topk(min(V, 6), dim=1).indices.view(R, T, -1)
    d = best[:, : T - 1].gather(2, torch.randint(0, best.shape[2], (R, T - 1, 1), generator=g))[..., 0].to(torch.int32)
    return x, d.contiguous(), torch.rand(R * T, generator=g), torch.rand(R, T - 1, generator=g)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("R,T,V", [(1, 2, 50), (1, 16, 5000), (7, 3, 1025), (64, 4, 700), (2, 9, 9001), (1, 5, 40000)])
def test_drafts(b, R, T, V, dt):
    for n, s in enumerate(SETTINGS[:20:2] + [SETTINGS[3]]):
        x, d, u, accept = speculative(R, T, V, n + T, DT[dt])
        d[0, 0] = (-1, V, 0)[n % 3]             # no token at all, or one far down
        got = b.sample_logits(x.cuda().view(R, T, V), u.cuda(), None, d.cuda(), temperature=s[0], top_k=s[1], top_p=s[2],
                              min_p=s[3], accept=accept.cuda())
        assert got[2].shape == (R, T - 1) and got[3].shape == (R,)
        check(got, x.double().numpy(), [s] * R, u, d, accept, R, T)


def test_draft_that_is_all_but_certain(b):
    """What remains beside a draft keeps its digits, down to a mass of e^-60 of it; and nothing may remain."""
    x = torch.randn(4, 500)
    x[:, 77] = 60.0
    x[2, :77] = x[2, 78:] = -math.inf
    d = torch.full((2, 1), 77, dtype=torch.int32)
    u, accept = torch.tensor([0.3, 0.3, 0.6, 0.6]), torch.zeros(2, 1)
    for s in ((1.0, 0, 1.0, 0.0), (1.0, 100, 1.0, 0.0), (2.0, 400, 1.0, 0.0), (1.0, 1, 1.0, 0.0), (1.0, 0, 0.9, 0.0),
              (0.0, 0, 1.0, 0.0)):
        got = b.sample_logits(x.cuda(), u.cuda(), None, d.cuda(), R=2, temperature=s[0], top_k=s[1], top_p=s[2],
                              min_p=s[3], accept=accept.cuda())
        check(got, x.double().numpy(), [s] * 2, u, d, accept, 2, 2)
        assert got[0][2].item() == -1 and got[3].tolist() == [1, 1]


@pytest.mark.parametrize("R,T,V", [(1, 1, 9000), (5, 4, 3001), (2, 16, 1500), (40, 2, 333)])
@pytest.mark.parametrize("dt", list(DT))
def test_under_rules(b, R, T, V, dt):
    g = np.random.default_rng(R + T + V)
    M = R * T
    x, d, u, accept = speculative(R, T, V, R + T, DT[dt]) if T > 1 else \
        (logits(M, V, DT[dt], 1), None, torch.rand(M), None)
    n = g.integers(0, 60, R)
    off = np.concatenate(([0], np.cumsum(n)))
    rules = dict(lr.NONE, history=g.integers(0, V, off[-1]).astype(np.int32), history_offsets=off,
                 n_prompt=(n // 2).astype(np.int32), repetition=(1 + g.random(R)).astype(np.float32),
                 frequency=g.random(R).astype(np.float32), presence=g.random(R).astype(np.float32),
                 bias_ids=g.integers(0, V, 4 * R).astype(np.int32),
                 bias_values=(3 * g.normal(size=4 * R)).astype(np.float32), bias_offsets=4 * np.arange(R + 1),
                 mask=g.integers(0, 2 ** 32, (3, (V + 31) // 32), dtype=np.uint32),
                 mask_index=g.integers(-1, 4, M).astype(np.int32))         # 3: nothing is allowed
    dev = b.LogitRules(**{k: torch.from_numpy(v.view(np.int32) if k == "mask" else v).cuda() for k, v in rules.items()})
    dn = d.numpy() if T > 1 else np.zeros((R, 0), np.int32)
    ruled = lr.ruled(x.float().numpy(), rules, dn, R, T)
    for s in SETTINGS[::3]:
        got = b.sample_logits(x.cuda(), u.cuda(), dev, gpu(d), R=R, temperature=s[0], top_k=s[1], top_p=s[2],
                              min_p=s[3], accept=gpu(accept))
        check(got, ruled.astype(np.float64), [s] * R, u, d, accept, R, T)


@pytest.mark.parametrize("s", [SETTINGS[0], SETTINGS[6], SETTINGS[18]])
def test_layouts_streams_and_graphs(b, s):
    R, T, V = 3, 4, 2500
    x, d, u, accept = (t.cuda() for t in speculative(R, T, V, 8))
    call = lambda lo: b.sample_logits(lo, u, None, d, R=R, temperature=s[0], top_k=s[1], top_p=s[2],  # noqa: E731
                                      min_p=s[3], accept=accept)
    want = call(x)
    wide = torch.full((R * T, V + 77), 50.0, device="cuda")
    wide[:, 3:3 + V] = x
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = call(x)
    side.synchronize()
    for got in (call(wide[:, 3:3 + V]), other, b.sample_logits(x.view(R, T, V), u.view(R, T), None, d, temperature=s[0],
                                                               top_k=s[1], top_p=s[2], min_p=s[3], accept=accept)):
        for a, w in zip(got, want):
            assert torch.equal(a, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(x)
    for i in range(4):
        x.copy_(x.roll(131, dims=1))
        u.copy_(torch.rand_like(u))
        graph.replay()
        eager = call(x)
        torch.cuda.synchronize()
        for a, w in zip(got, eager):
            assert torch.equal(a, w)


def test_rows_beyond_32_bit_offsets(b):
    """Rows 2^31 + 2^20 elements apart."""
    V, far = 5000, (1 << 31) + (1 << 20)
    buf = torch.empty(far + V, dtype=torch.bfloat16, device="cuda")
    rows = torch.as_strided(buf, (2, V), (far, 1))
    x = logits(2, V, torch.bfloat16, 9)
    rows.copy_(x)
    u = torch.tensor([0.4, 0.8])
    for s in (SETTINGS[0], SETTINGS[6]):
        got = b.sample_logits(rows, u.cuda(), R=2, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        check(got, x.double().numpy(), [s] * 2, u)


def test_most_rows(b):
    """4096 rows, whose candidates' places pass 32 bits of bytes."""
    R, T, V = 1024, 4, 151936
    one = logits(8, V, torch.bfloat16, 10)
    x = one.cuda().repeat(R * T // 8, 1)
    u = torch.rand(R * T)
    d = torch.randint(0, V, (R, T - 1), dtype=torch.int32)
    for s in ((0.9, 50, 0.95, 0.0), (1.0, 0, 1.0, 0.0)):
        got = b.sample_logits(x, u.cuda(), None, d.cuda(), R=R, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        keep = [0, 1, 2, 3, 2000, 2001, 2002, 2003, 4092, 4093, 4094, 4095]
        check([None if t is None else t[keep] for t in got], one.double().numpy()[[r % 8 for r in keep]], [s] * 12,
              u[keep])


def test_longest_rows(b):
    """2^24 tokens."""
    V = 1 << 24
    x = torch.randn(1, V)
    x[0, 12345678] = 11.0
    x[0, 16777215] = 12.0
    u = torch.tensor([0.9999])
    for s in ((0.2, 0, 1.0, 0.0), (0.2, 0, 0.9, 0.0), (0.3, 20, 1.0, 0.0)):
        got = b.sample_logits(x.cuda(), u.cuda(), R=1, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        check(got, x.double().numpy(), [s], u)


@pytest.mark.parametrize("M,V", [(40, 1025), (2, 33), (1, 3001), (9, 9000)])
def test_rows_without_a_token(b, M, V):
    """Rows of which nothing is allowed leave their neighbours, and what lies behind the workspace, as they are."""
    x = logits(M, V, torch.float32, M)
    x[::2] = -math.inf
    x[::4, ::3] = math.nan
    u = torch.linspace(0, 0.999, M)
    L, dev, du = b.load_library(), x.cuda(), u.cuda()
    need = L.sample_logits_workspace_bytes(M, 1, V)
    for s in ((0.0, 0, 1.0, 0.0), (1.0, 1, 1.0, 0.0), (1.0, 5, 0.9, 0.0), (1.0, 0, 0.9, 0.1), (1.0, 0, 1.0, 0.0)):
        ids, probs = torch.empty(M, dtype=torch.int32).cuda(), torch.empty(M).cuda()
        ws = torch.full((need + 65536,), 0xA5, dtype=torch.uint8).cuda()
        st = L.sample_logits_rows(dev.data_ptr(), V, 2, None, M, 1, V, None, b._SAMPLING.pack(0, 0, 0, 0, *s),
                                  du.data_ptr(), None, ids.data_ptr(), probs.data_ptr(), None, None,
                                  ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        check((ids, probs, None, None), x.double().numpy(), [s] * M, u)
        assert (ids[::2] == -1).all() and bool((ws[need:] == 0xA5).all())


@pytest.mark.parametrize("V", [5000, 9000, 40000])
@pytest.mark.parametrize("shape", ["flat", "shelf"])
def test_many_candidates(b, V, shape):
    """Thousands of candidates, of which few or most are kept, with and without drafts."""
    R, T = 3, 2
    g = torch.Generator().manual_seed(V)
    x = torch.randn(R * T, V, generator=g)
    if shape == "shelf":
        x[:, : V // 4] += 6.0                   # most of the mass in a quarter of the tokens
    u = torch.rand(R * T, generator=g)
    d = x.topk(3, dim=1).indices.view(R, T, 3)[:, : T - 1, 1].to(torch.int32).contiguous()
    accept = torch.rand(R, T - 1, generator=g)
    for s in ((1.0, 0, 0.3, 0.0), (1.0, 0, 0.9, 0.0), (0.5, 0, 0.999, 0.0), (1.0, V // 3, 1.0, 0.0),
              (1.0, V - 1, 0.6, 0.0), (3.0, 4200, 0.99, 0.01), (1.0, 0, 0.7, 0.2)):
        kw = dict(R=R, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        check(b.sample_logits(x.cuda(), u.cuda(), None, d.cuda(), **kw), x.double().numpy(), [s] * R, u, R=R, T=T)
        check(b.sample_logits(x.cuda(), u.cuda(), None, d.cuda(), accept=accept.cuda(), **kw), x.double().numpy(),
              [s] * R, u, d, accept, R, T)


@pytest.mark.parametrize("n", [300, 700, 5000])
def test_fewer_tokens_than_top_k(b, n):
    """A row that holds no top_k tokens above -infinity: top_p and min_p still hold."""
    V = 9000
    x = torch.full((4, V), -math.inf)
    x[:, 1000:1000 + n] = torch.randn(4, n, generator=torch.Generator().manual_seed(n))
    u = torch.tensor([0.1, 0.5, 0.9, 0.999])
    for s in ((1.0, n + 50, 0.6, 0.0), (2.0, 8000, 0.9, 0.1), (1.0, n + 1, 1.0, 0.2), (1.0, n, 0.3, 0.0)):
        got = b.sample_logits(x.cuda(), u.cuda(), R=4, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
        check(got, x.double().numpy(), [s] * 4, u)


def test_binding_refusals(b):
    x, d, u, accept = (t.cuda() for t in speculative(2, 3, 100, 1))
    ok = dict(logits=x, uniforms=u, draft_ids=d, R=2)
    bad = [(dict(uniforms=u[:5]), ValueError), (dict(uniforms=u.double()), TypeError), (dict(uniforms=u.cpu()), TypeError),
           (dict(draft_ids=None), ValueError), (dict(R=None), ValueError), (dict(R=4), ValueError),
           (dict(accept=accept[:1]), ValueError), (dict(temperature=-1.0), RuntimeError),
           (dict(temperature=float("nan")), RuntimeError), (dict(top_k=-1), RuntimeError), (dict(top_p=1.5), RuntimeError),
           (dict(min_p=-0.1), RuntimeError), (dict(temperature=torch.ones(3).cuda()), ValueError),
           (dict(top_k=torch.ones(2).cuda()), TypeError), (dict(top_p=torch.ones(2)), TypeError),
           (dict(top_k=2.5), TypeError), (dict(logits=x.double()), TypeError)]
    for kw, err in bad:
        with pytest.raises(err):
            b.sample_logits(**{**ok, **kw})
    with pytest.raises(ValueError):
        b.sample_logits(x, u, R=6, accept=accept)
