"""Rules and verification where a wave walks several chunks of 1024 tokens, as
it does in batches (GPU): what a wave carries from chunk to chunk (its bound,
its candidates, its running maximum and sum), the alternating loads and the
write behind them, slices as long as they get, and rows cut into more lists
than the merge holds at once.  Each case first checks, from the lists that a
call leaves in its workspace, that its waves do take that many chunks.

Selections are exact.  Tolerances of lse and p as in test_gpu_logit_rules: 90 u
+ 3 u |lse| (u = 2^-24), and p's 190 u + 3 u |z|."""
import numpy as np
import pytest
import torch

from oracle import logit_rules as lr
from tests.test_gpu_logit_rules import U, dev, device_rules, make, same

pytestmark = pytest.mark.gpu
CHUNK = 1024
INF = float("inf")


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def lists_per_row(b, logits, rules, R, T, k):
    """How many lists each row of such a call is cut into: the call writes M *
    n_lists * max(k, 1) 64-bit keys to the front of its workspace."""
    M, V = logits.shape
    L = b.load_library()
    code = {torch.float32: 2, torch.float16: 0, torch.bfloat16: 1}[logits.dtype]
    need = L.logit_rules_verify_workspace_bytes(R, T, V, k)
    mark = 0x5A5A5A5A5A5A5A5A                          # the key of no token: its id would lie outside
    ws = torch.full((need // 8,), mark, dtype=torch.int64, device="cuda")
    new = lambda n, dt: torch.empty(max(n, 1), dtype=dt, device="cuda")  # noqa: E731
    f, i = torch.float32, torch.int32
    o = [new(M, f), new(M, i), new(M * k, i), new(M * k, f), new(R, i)]
    d = torch.zeros(R * max(T - 1, 1), dtype=i, device="cuda")
    st = L.logit_rules_verify(logits.data_ptr(), V, code, d.data_ptr(), None, None, R, T, V,
                              None if rules is None else rules.packed, k, 1.0, o[0].data_ptr(), o[1].data_ptr(),
                              o[2].data_ptr() if k else None, o[3].data_ptr() if k else None, None, None,
                              o[4].data_ptr(), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    area = ws[: M * ((V + CHUNK - 1) // CHUNK + 8) * max(k, 1)]
    n = int((area != mark).sum())
    assert n % (M * max(k, 1)) == 0
    return n // (M * max(k, 1))


def chunks_per_wave(b, logits, rules, R, T, k):
    n = lists_per_row(b, logits, rules, R, T, k)
    return -(-((logits.shape[1] + CHUNK - 1) // CHUNK) // n)


def check(got, x, drafts, dp, un, R, T, k, tau):
    """got against a stable sort and sums in 64 bits of the ruled logits x
    (binary32, on the GPU)."""
    lmax, amax, tids, tlog, pdr, nacc, lse = got
    M, V = x.shape
    x = torch.where(torch.isnan(x), -INF, x)
    order = torch.sort(x, dim=1, descending=True, stable=True)
    n = max(k, 1)
    val = order.values[:, :n]
    ids = torch.where(val > -INF, order.indices[:, :n], -1).int()
    assert torch.equal(amax, ids[:, 0]) and torch.equal(lmax, val[:, 0])
    if k:
        assert torch.equal(tids, ids), torch.nonzero(tids != ids)[:5]
        assert torch.equal(tlog, val)
    z = x.double()
    m = z.max(dim=1, keepdim=True).values
    m0 = torch.where(m > -INF, m, 0.0)
    if lse is not None:
        want = (m / tau + torch.log(torch.exp((z - m0) / tau).sum(1, keepdim=True)))[:, 0]
        ok = (lse.double() - want).abs() <= 90 * U + 3 * U * want.abs()
        assert bool((ok | ((want == -INF) & (lse == -INF))).all())
    if T == 1:
        return
    rows = torch.arange(M, device="cuda").view(R, T)[:, : T - 1]
    d = drafts.long()
    if dp is not None:
        inside = (d >= 0) & (d < V)
        zd = z[rows, d.clamp(0, V - 1)]
        e = torch.exp(((val.double() if k else z) - m0) / tau).sum(dim=1)[rows]
        among = (ids.view(R, T, n)[:, : T - 1] == drafts[..., None]).any(dim=2) if k else zd > -INF
        want = torch.where(inside & among, torch.exp((zd - m0[rows, 0]) / tau) / e, 0.0)
        share = torch.where(want > 0, -torch.log(want.clamp(min=1e-300)) + np.log(V) + 1, 0.0)
        off = (pdr.double() - want).abs()
        assert bool((off <= want * (190 * U + 3 * U * share) + 2.0 ** -149).all())
        ok = un * dp < pdr
    else:
        ok = ids[:, 0].view(R, T)[:, : T - 1] == drafts
    assert torch.equal(nacc, ok.int().cumprod(dim=1).sum(dim=1).int())


def near(x, R, T, seed):
    """Drafts among a row's best, some past the vocabulary."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    V = x.shape[1]
    best = torch.topk(torch.where(torch.isnan(x), -INF, x), min(4, V), dim=1).indices.view(R, T, -1)[:, : T - 1]
    pick = (torch.rand(R, T - 1, 1, generator=g, device="cuda") ** 3 * best.shape[2]).long()
    d = best.gather(2, pick)[..., 0].int().contiguous()
    d[:, -1:][::3] = V
    return d


def uniforms(R, T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(R, T - 1, generator=g, device="cuda") for _ in range(2))


# R, T and the chunks that a wave takes of rows of 70001 tokens (69 chunks, the
# last one of 369)
BATCHES = [(64, 4, 4), (32, 4, 2), (64, 2, 2), (32, 16, 8), (32, 11, 8), (128, 3, 4), (9, 1, 1)]
V0 = 70001


@pytest.mark.parametrize("R,T,per", BATCHES)
def test_rules_over_several_chunks(b, R, T, per):
    for bias, history, dt in ((5, 200, torch.float32), (9000 // R, 60, torch.float16)):
        logits, rules, drafts = make(R, T, V0, R + T, bias=bias, history=history)
        # words of the history and biases at the ends of chunks and slices
        rules["history"][3::11] = (rules["history"][3::11] // CHUNK * CHUNK - 1).clip(0, V0 - 1)
        rules["history"][4::13] = V0 - 1
        apart = len(rules["bias_ids"]) > 2047
        assert apart == (bias > 5)                     # both layouts of a token's words
        t = torch.from_numpy(logits).to(dt)
        r, d = device_rules(b, rules), dev(drafts) if T > 1 else None
        want = lr.ruled(t.float().numpy(), rules, drafts, R, T)
        x = t.cuda()
        for k in (0, 16):
            assert chunks_per_wave(b, x, r, R, T, k) == per
        out = b.apply_logit_rules(x, r, d, R=R)
        same(out, torch.from_numpy(want).to(dt).float().numpy())
        ruled = torch.from_numpy(want).cuda()
        if T > 1:
            assert torch.equal(x.cpu(), t)
        check(b.verify_logits(x, r, d, R=R, top_k=16, want_lse=True), ruled, d, None, None, R, T, 16, 1.0)
        check(b.verify_logits(x, r, d, R=R, want_lse=True, temperature=0.7), ruled, d, None, None, R, T, 0, 0.7)
        if T > 1:
            dp, un = uniforms(R, T, 1)
            for k in (0, 1, 9):
                check(b.verify_logits(x, r, d, dp, un, R=R, top_k=k, temperature=1.3), ruled, d, dp, un, R, T, k, 1.3)
        # in place, in strided rows between others
        big = torch.full((R * T, V0 + 7), 3.0, dtype=dt, device="cuda")
        big[:, 5: 5 + V0] = x
        b.apply_logit_rules(big[:, 5: 5 + V0], r, d, R=R, out=big[:, 5: 5 + V0])
        assert torch.equal(torch.nan_to_num(big[:, 5: 5 + V0]), torch.nan_to_num(out))
        assert bool((big[:, :5] == 3).all()) and bool((big[:, 5 + V0:] == 3).all())


KINDS = ["equal", "ascending", "descending", "few_values", "one_lane", "sparse", "saw", "steps", "late", "infinite",
         "nan"]


def order(kind, M, V):
    g = torch.Generator(device="cuda").manual_seed(M + len(kind))
    v = torch.arange(V, device="cuda", dtype=torch.float32)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if kind == "equal":
        return torch.full((M, V), 1.5, device="cuda")
    if kind == "ascending":
        return v.repeat(M, 1)
    if kind == "descending":
        return -v.repeat(M, 1)
    if kind == "few_values":                           # ties of the k-th value in every chunk
        return torch.randint(0, 3, (M, V), generator=g, device="cuda").float()
    if kind == "one_lane":
        x = rnd(M, V)
        x[:, 5::64] += 50
        return x
    if kind == "sparse":                               # a handful above -infinity, none in many chunks
        x = torch.full((M, V), -INF, device="cuda")
        for m in range(M):
            n = m % 9
            x[m, torch.randint(0, V, (n,), generator=g, device="cuda")] = rnd(n)
        return x
    if kind == "saw":                                  # descending in a chunk, each chunk above the one before
        return ((v // CHUNK) * CHUNK - v % CHUNK).repeat(M, 1)
    if kind == "steps":                                # a chunk holds one value, larger in later chunks
        return (v // CHUNK).repeat(M, 1)
    x = rnd(M, V)
    if kind == "late":                                 # the best in the last, partial chunk
        x[:, -20:] += 100
    elif kind == "infinite":
        x[torch.rand(M, V, generator=g, device="cuda") < 0.001] = INF
        x[::3] = rnd(1, V)
        x[::3, V // 2] = INF
    else:
        x[torch.rand(M, V, generator=g, device="cuda") < 0.5] = float("nan")
        x[0], x[1, : V - 1] = float("nan"), float("nan")
    return x


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("R,T,per", [(64, 4, 4), (32, 4, 2), (32, 16, 8)])
def test_hard_orders_over_several_chunks(b, R, T, per, kind):
    for dt in (torch.float32, torch.float16):
        x = order(kind, R * T, V0).to(dt)
        d = near(x.float(), R, T, 3)
        dp, un = uniforms(R, T, 2)
        for k in (0, 1, 5, 16):
            assert chunks_per_wave(b, x, None, R, T, k) == per
            infinite = kind == "infinite" or dt == torch.float16 and kind in ("ascending", "saw")   # past 65504
            got = b.verify_logits(x, None, d, R=R, top_k=k, want_lse=not infinite)
            check(got, x.float(), d, None, None, R, T, k, 1.0)
            if not infinite:
                got = b.verify_logits(x, None, d, dp, un, R=R, top_k=k, temperature=0.9)
                check(got, x.float(), d, dp, un, R, T, k, 0.9)


def test_masks_over_several_chunks(b):
    """Masks that allow nothing, one token, or nothing in most chunks, and
    anything in the places that they refuse."""
    R, T = 64, 4
    M, W = R * T, (V0 + 31) // 32
    g = torch.Generator(device="cuda").manual_seed(0)
    allowed = torch.zeros(M, W * 32, dtype=torch.bool, device="cuda")
    for m in range(1, M):
        n = (0, 1, 5, 40)[m % 4]
        allowed[m, torch.randint(0, V0, (n,), generator=g, device="cuda")] = True
    allowed[5, V0 - 1] = True
    allowed[:, V0:] = True                             # bits past the vocabulary are nobody's
    bits = allowed.view(M, W, 32).long() << torch.arange(32, device="cuda")
    words = bits.sum(dim=2)
    mask = torch.where(words >= 2 ** 31, words - 2 ** 32, words).int().contiguous()
    x = torch.randn(M, V0, generator=g, device="cuda")
    clean = torch.where(allowed[:, :V0], x, -INF)
    for bad in (float("nan"), INF, -INF, torch.finfo(torch.float32).min):
        y = torch.where(allowed[:, :V0], x, bad)
        r = b.LogitRules(mask=mask)
        d = near(clean, R, T, 1)
        dp, un = uniforms(R, T, 4)
        assert torch.equal(b.apply_logit_rules(y, r, d, R=R), clean)
        for k in (0, 16):
            check(b.verify_logits(y, r, d, R=R, top_k=k, want_lse=True), clean, d, None, None, R, T, k, 1.0)
            check(b.verify_logits(y, r, d, dp, un, R=R, top_k=k), clean, d, dp, un, R, T, k, 1.0)


@pytest.mark.parametrize("R,T,V", [(1, 1, 8192), (2, 1, 20000), (64, 4, V0)])
def test_the_longest_slices(b, R, T, V):
    """8192 tokens a slice, counts and bias entries in words apart, and top-k
    buffers: 72 KB of LDS, the most that a call takes."""
    nb = 2100
    g = np.random.default_rng(5)
    logits, rules, drafts = make(R, T, V, 2, history=100, bias=0)
    rules["bias_ids"] = g.integers(0, V, nb).astype(np.int32)
    rules["bias_values"] = g.normal(0, 4, nb).astype(np.float32)
    rules["bias_offsets"] = np.linspace(0, nb, R + 1).astype(np.int64)
    x, r = dev(logits), device_rules(b, rules)
    d = dev(drafts) if T > 1 else None
    # 8 waves, of T rows: a slice of 8 chunks is 8 / T lists of every row, as V is
    slices = (V + 8191) // 8192
    assert lists_per_row(b, x, r, R, T, 16) == slices * (8 // T)
    want = lr.ruled(logits, rules, drafts, R, T)
    same(b.apply_logit_rules(x, r, d, R=R), want)
    ruled = torch.from_numpy(want).cuda()
    for k in (0, 16):
        check(b.verify_logits(x, r, d, R=R, top_k=k, want_lse=True), ruled, d, None, None, R, T, k, 1.0)


@pytest.mark.parametrize("R,T,V,dt", [(1, 16, 300001, torch.float32), (1, 1, 300001, torch.float32),
                                      (1, 3, 600000, torch.float16), (1, 1, 1 << 24, torch.float32)])
def test_rows_of_very_many_lists(b, R, T, V, dt):
    """More lists than the merge's lanes hold the first keys of at once (256)."""
    for kind in ("few_values", "late", "ascending", "descending", "sparse"):
        x = order(kind, R * T, V)
        x = (x / 16 if dt == torch.float16 and V > 65504 else x).to(dt)
        d = near(x.float(), R, T, 3) if T > 1 else None
        for k in (0, 1, 16):
            assert lists_per_row(b, x, None, R, T, k) > 256
            check(b.verify_logits(x, None, d, R=R, top_k=k, want_lse=True), x.float(), d, None, None, R, T, k, 1.0)


def test_graphs_over_several_chunks(b):
    R, T = 64, 4
    logits, rules, drafts = make(R, T, V0, 9)
    r, x, d = device_rules(b, rules), dev(logits), dev(drafts)

    def run():
        return [b.apply_logit_rules(x, r, d, R=R)] + \
            [t for t in b.verify_logits(x, r, d, R=R, top_k=16, want_lse=True) if t is not None]
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for rep in range(3):
        x.normal_(generator=torch.Generator(device="cuda").manual_seed(rep))
        want = run()
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip(out, want):
            assert torch.equal(u, v)
