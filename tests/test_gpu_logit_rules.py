"""Rules on logits and verification under them (GPU): the ruled logits bit for
bit in the documented binary32 order and against the formula in 64 bits, and
the verification against the plain form on those logits.

Tolerances, u = 2^-24.  Ruled values: one rounding per step, u times the sum of
the steps' magnitudes, then half a step of the output's type.  lse: a term's
exponent z = (x - max) log2(e) / tau carries 3 u |z| and the exponential 2 u,
weighted by the terms' shares at most 3 u (ln V + 1) + 2 u, and the sums' 40
roundings: below 90 u for V <= 2^20, plus 3 u |lse| for max / tau, the sum and
the final rounding.  p: twice the former plus 3 u |z_d| of its own exponent."""
import numpy as np
import pytest
import torch

from oracle import logit_rules as lr

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
INT = ("history", "n_prompt", "bias_ids", "mask", "mask_index")


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def make(R, T, V, seed, history=200, bias=5, mask="index", penalties=("repetition", "frequency", "presence"),
         allowed=0.3):
    g = np.random.default_rng(seed)
    M = R * T
    logits = g.normal(0, 3, (M, V)).astype(np.float32)
    rules = dict(lr.NONE)
    if history:
        n = g.integers(0, history + 1, R)
        if R > 1:
            n[R // 2] = 0                              # a request without any history
        rules["history_offsets"] = np.concatenate(([0], np.cumsum(n))).astype(np.int64)
        words = (V * g.random(int(n.sum()) + 3) ** 3).astype(np.int32)
        words[::17] = V + 5                            # ids outside the vocabulary are ignored
        words[5::23] = -1
        rules["history"] = words
        rules["n_prompt"] = g.integers(0, history + 1, R).astype(np.int32)     # some beyond the history's end
    for name in penalties:
        rules[name] = (g.random(R) + (0.5 if name == "repetition" else -0.3)).astype(np.float32)
    if bias:
        n = g.integers(0, bias + 1, R)
        rules["bias_offsets"] = np.concatenate(([0], np.cumsum(n))).astype(np.int64)
        ids = g.integers(-2, V + 2, int(n.sum())).astype(np.int32)
        ids[1::4] = ids[:1] if len(ids) else 0         # the same id again
        rules["bias_ids"], rules["bias_values"] = ids, g.normal(0, 4, len(ids)).astype(np.float32)
    if mask:
        n = M if mask == "rows" else max(1, M // 2)
        W = (V + 31) // 32
        bits = np.zeros((n, W * 32), bool)
        bits[:, :V] = g.random((n, V)) < allowed
        bits[0] = False                                # a mask that leaves nothing
        rules["mask"] = np.packbits(bits.reshape(n, W, 32), axis=2, bitorder="little").view(np.uint32)[..., 0]
        if mask == "index":
            rules["mask_index"] = g.integers(-1, n, M).astype(np.int32)
            rules["mask_index"][0] = 0
    drafts = np.stack([g.permutation(V)[: T - 1] if V >= T - 1 else g.integers(0, V, T - 1) for _ in range(R)]) \
        if T > 1 else np.zeros((R, 0))
    drafts = drafts.astype(np.int32)
    if T > 2:
        drafts[:, 1] = drafts[:, 0]                    # the same draft twice
    if T > 3:
        drafts[0, 2] = V                               # an id outside the vocabulary
    return logits, rules, drafts


def device_rules(b, rules):
    kw = {k: None if v is None else torch.from_numpy(v.view(np.int32) if k == "mask" else v).cuda()
          for k, v in rules.items()}
    return b.LogitRules(**kw)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def same(got, want):
    """Equal values; NaN with NaN, and zeros of either sign."""
    got = got.float().cpu().numpy()
    ok = (got == want) | (np.isnan(got) & np.isnan(want))
    assert ok.all(), (np.argwhere(~ok)[:5], got[~ok][:5], want[~ok][:5])


SHAPES = [(1, 1, 1), (1, 1, 33), (2, 3, 31), (3, 1, 1000), (1, 16, 1023), (4, 4, 1024), (2, 5, 1025), (5, 2, 4097),
          (1, 2, 8192), (2, 16, 8193), (1, 3, 20011), (70, 4, 2050), (1, 1, 151936), (3, 4, 151936)]


@pytest.mark.parametrize("R,T,V", SHAPES)
def test_apply(b, R, T, V):
    for mask in ("index", "rows", None):
        logits, rules, drafts = make(R, T, V, R + T + V, mask=mask)
        got = b.apply_logit_rules(dev(logits), device_rules(b, rules), dev(drafts) if T > 1 else None, R=R)
        same(got, lr.ruled(logits, rules, drafts, R, T))
    want = lr.ruled(logits, rules, drafts, R, T, np.float64)
    off = np.abs(got.cpu().numpy().astype(np.float64) - want)
    # the steps' magnitudes: at most 2 |l|, count * 0.7, 0.7 and the bias
    bound = 2 * np.abs(logits) + 0.7 * 216 + 0.7 + 20
    assert np.all(off <= 5 * U * bound)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("R,T,V", [(1, 1, 1001), (2, 4, 5000), (3, 2, 1024)])
def test_apply_in_16_bits(b, R, T, V, dt):
    logits, rules, drafts = make(R, T, V, 5)
    x = torch.from_numpy(logits).to(DT[dt])
    got = b.apply_logit_rules(x.cuda(), device_rules(b, rules), dev(drafts) if T > 1 else None, R=R)
    want = torch.from_numpy(lr.ruled(x.float().numpy(), rules, drafts, R, T)).to(DT[dt])      # rounded once
    assert got.dtype == DT[dt]
    same(got, want.float().numpy())


def test_each_rule_alone(b):
    R, T, V = 3, 4, 3000
    for kw in (dict(penalties=("repetition",), bias=0, mask=None), dict(penalties=("frequency",), bias=0, mask=None),
               dict(penalties=("presence",), bias=0, mask=None), dict(penalties=(), bias=0, mask="rows"),
               dict(penalties=(), bias=9, mask=None, history=0), dict(history=0, bias=0, mask=None),
               dict(penalties=(), bias=0, mask=None, history=0), dict(penalties=(), history=50, bias=3)):
        logits, rules, drafts = make(R, T, V, 12, **kw)
        if kw.get("history", 200) == 0 and "penalties" not in kw:
            rules["history"] = rules["history_offsets"] = None     # drafts alone count
        got = b.apply_logit_rules(dev(logits), device_rules(b, rules), dev(drafts), R=R)
        same(got, lr.ruled(logits, rules, drafts, R, T))
    x = dev(logits)
    assert torch.equal(b.apply_logit_rules(x, None, dev(drafts), R=R), x)


def test_long_history(b):
    """A history longer than one round of a workgroup's loads, one token of it
    tens of thousands of times, and one without n_prompt."""
    R, T, V = 2, 3, 9000
    logits, rules, drafts = make(R, T, V, 3, history=70000, bias=0, mask=None)
    rules["history"][: rules["history"].size // 2] = 8191
    for n_prompt in (rules["n_prompt"], None):
        rules["n_prompt"] = n_prompt
        got = b.apply_logit_rules(dev(logits), device_rules(b, rules), dev(drafts), R=R)
        same(got, lr.ruled(logits, rules, drafts, R, T))


@pytest.mark.parametrize("n,nb", [((1 << 20) + 5, 40), (300, 4000), (300, 2047), ((1 << 20) - 32, 2047)])
def test_counts_and_entries_too_many_for_one_word(b, n, nb):
    """On both sides of the lengths up to which a token's count and its bias
    entry share a word; one token fills the history, and the last entry of an
    id holds."""
    R, T, V = 1, 3, 3000
    g = np.random.default_rng(n + nb)
    logits, rules, drafts = make(R, T, V, 1, history=0, bias=0, mask=None)
    rules["history"] = np.full(n, 17, np.int32)
    rules["history"][: n // 3] = g.integers(0, V, n // 3)
    rules["history_offsets"] = np.array([0, n], np.int64)
    rules["n_prompt"] = np.array([n // 5], np.int32)
    rules["bias_ids"] = g.integers(0, V, nb).astype(np.int32)
    rules["bias_values"] = g.normal(0, 4, nb).astype(np.float32)
    rules["bias_offsets"] = np.array([0, nb], np.int64)
    drafts[0, :] = 17
    want = logits.copy()
    made = np.bincount(rules["history"][n // 5:], minlength=V)
    seen = np.bincount(rules["history"], minlength=V) > 0
    last = dict(zip(rules["bias_ids"].tolist(), rules["bias_values"]))
    rep, freq, pres = (rules[k][0] for k in ("repetition", "frequency", "presence"))
    for t in range(T):
        row, count = want[t], made.copy()
        count[17] += t
        row[seen] = np.where(row[seen] > 0, row[seen] / rep, row[seen] * rep)
        m = count > 0
        row[m] = row[m] - freq * count[m].astype(np.float32)
        row[m] = row[m] - pres
        for v, x in last.items():
            row[v] = row[v] + np.float32(x)
    same(b.apply_logit_rules(dev(logits), device_rules(b, rules), dev(drafts), R=R), want)


def test_verify_with_the_longest_slices(b):
    """Words apart, whole slices and top-k lists: the most LDS a call takes."""
    R, T, V, nb = 60, 4, 20000, 3000
    g = np.random.default_rng(5)
    logits, rules, drafts = make(R, T, V, 2, history=100, bias=0)
    rules["bias_ids"] = g.integers(0, V, nb).astype(np.int32)
    rules["bias_values"] = g.normal(0, 4, nb).astype(np.float32)
    rules["bias_offsets"] = np.linspace(0, nb, R + 1).astype(np.int64)
    x = lr.ruled(logits, rules, drafts, R, T)
    got = b.verify_logits(dev(logits), device_rules(b, rules), dev(drafts), R=R, top_k=16, want_lse=True)
    check_verify(got, x, drafts, None, None, R, T, 16, 1.0, True)
    same(b.apply_logit_rules(dev(logits), device_rules(b, rules), dev(drafts), R=R), x)


def test_offsets_outside_are_clamped(b):
    logits, rules, drafts = make(2, 2, 500, 3)
    n, m = len(rules["history"]), len(rules["bias_ids"])
    rules["history_offsets"] = np.array([-5, 40, n + 100], np.int64)
    rules["bias_offsets"] = np.array([-1, 1, m + 9], np.int64)
    rules["mask_index"][1] = 10 ** 6                   # past the masks: nothing is allowed
    got = b.apply_logit_rules(dev(logits), device_rules(b, rules), dev(drafts), R=2)
    want = lr.ruled(logits, rules, drafts, 2, 2)
    assert np.isinf(want[1]).all()
    same(got, want)
    rules["history_offsets"] = np.array([60, 40, 20], np.int64)
    same(b.apply_logit_rules(dev(logits), device_rules(b, rules), dev(drafts), R=2),
         lr.ruled(logits, rules, drafts, 2, 2))


@pytest.mark.parametrize("V", [100, 1025, 8193])
def test_strides_in_place_and_rows_behind(b, V):
    R, T = 2, 3
    logits, rules, drafts = make(R, T, V, 4)
    want = lr.ruled(logits, rules, drafts, R, T)
    r, d = device_rules(b, rules), dev(drafts)
    big = torch.full((R * T + 1, V + 9), 5.0, device="cuda")
    view = big[: R * T, 3: 3 + V]
    view.copy_(dev(logits))
    out = torch.full((R * T + 1, V + 2), 6.0, device="cuda")
    b.apply_logit_rules(view, r, d, R=R, out=out[: R * T, 1: 1 + V])
    same(out[: R * T, 1: 1 + V], want)
    same(view, logits)
    b.apply_logit_rules(view, r, d, R=R, out=view)
    same(view, want)
    view.fill_(5.0)
    out[: R * T, 1: 1 + V] = 6.0
    assert torch.equal(big, torch.full_like(big, 5.0)) and torch.equal(out, torch.full_like(out, 6.0))
    # a mask with words behind those the vocabulary needs
    wide = torch.zeros(rules["mask"].shape[0], rules["mask"].shape[1] + 3, dtype=torch.int32, device="cuda")
    wide[:, : rules["mask"].shape[1]] = torch.from_numpy(rules["mask"].view(np.int32)).cuda()
    kw = {k: None if v is None else torch.from_numpy(v).cuda() for k, v in rules.items() if k != "mask"}
    same(b.apply_logit_rules(dev(logits).view(R, T, V), b.LogitRules(mask=wide, **kw), d).view(R * T, V), want)


def test_masked_places_may_hold_anything(b):
    logits, rules, drafts = make(2, 2, 2000, 6, mask="rows")
    clean = lr.ruled(logits, rules, drafts, 2, 2)
    refused = np.isneginf(clean)
    for v in (np.nan, np.inf, -np.inf, np.finfo(np.float32).min, np.finfo(np.float32).max):
        x = logits.copy()
        x[refused] = v
        r = device_rules(b, rules)
        same(b.apply_logit_rules(dev(x), r, dev(drafts), R=2), clean)
        a, c = (b.verify_logits(dev(y), r, dev(drafts), R=2, top_k=5, want_lse=True) for y in (x, logits))
        for u, w in zip(a, c):
            assert u is None or torch.equal(u, w)


def check_verify(got, x, drafts, dp, un, R, T, k, tau, lse):
    """got against the plain form on the ruled logits x (binary32)."""
    lmax, amax, tids, tlog, pdr, nacc, lse_got = (None if t is None else t.cpu().numpy() for t in got)
    M, V = x.shape
    for m in range(M):
        ids, val = lr.top(x[m], 1)
        assert (amax[m], lmax[m]) == (ids[0], val[0]), m
        if k:
            ids, val = lr.top(x[m], k)
            assert np.array_equal(tids[m], ids) and np.array_equal(tlog[m], val), (m, tids[m], ids)
        if lse:
            want = lr.lse64(x[m], tau)
            assert lse_got[m] == want or abs(lse_got[m] - want) <= 90 * U + 3 * U * abs(want), (m, lse_got[m], want)
    for i in range(R):
        n = 0
        ok = True
        for t in range(T - 1):
            m, d = i * T + t, int(drafts[i, t])
            if dp is not None:
                want = lr.probability64(x[m], d, tau, k)
                # |z_d| is at most -ln p plus the logarithm of the terms that share it
                z = -np.log(want) + np.log(V) + 1 if want > 0 else 0
                assert abs(pdr[i, t] - want) <= want * (190 * U + 3 * U * z) + 2.0 ** -149, (i, t, pdr[i, t], want)
                ok = ok and np.float32(un[i, t]) * np.float32(dp[i, t]) < pdr[i, t]
            else:
                ok = ok and amax[m] == d
            n += ok
        assert nacc[i] == n


def near_drafts(x, drafts, R, T, seed):
    """Drafts that are often among a row's best."""
    g = np.random.default_rng(seed)
    d = drafts.copy()
    for i in range(R):
        for t in range(T - 1):
            best = [int(v) for v in lr.top(x[i * T + t], 3)[0] if v >= 0]
            if best and g.random() < 0.8:
                d[i, t] = best[int(len(best) * g.random() ** 3)]
    return d


@pytest.mark.parametrize("k", [0, 1, 7, 16])
@pytest.mark.parametrize("R,T,V", SHAPES)
def test_verify(b, R, T, V, k):
    k = min(k, V)
    tau = (1.0, 0.6, 1.7)[(R + T + k) % 3]
    logits, rules, drafts = make(R, T, V, R * T + V + k)
    drafts = near_drafts(lr.ruled(logits, rules, drafts, R, T), drafts, R, T, k)
    x = lr.ruled(logits, rules, drafts, R, T)
    g = np.random.default_rng(k)
    dp, un = g.random((2, R, T - 1)).astype(np.float32)
    r = device_rules(b, rules)
    d = dev(drafts) if T > 1 else None
    got = b.verify_logits(dev(logits), r, d, R=R, top_k=k, temperature=tau, want_lse=True)
    check_verify(got, x, drafts, None, None, R, T, k, tau, True)
    if T > 1:
        got = b.verify_logits(dev(logits), r, d, dev(dp), dev(un), R=R, top_k=k, temperature=tau)
        check_verify(got, x, drafts, dp, un, R, T, k, tau, False)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_verify_in_16_bits(b, dt):
    """16-bit logits tie often: ranks go to the lower token."""
    R, T, V = 3, 4, 12345
    logits, rules, drafts = make(R, T, V, 8)
    t = torch.from_numpy(logits).to(DT[dt])
    x = lr.ruled(t.float().numpy(), rules, drafts, R, T)
    got = b.verify_logits(t.cuda(), device_rules(b, rules), dev(drafts), R=R, top_k=16, want_lse=True)
    check_verify(got, x, drafts, None, None, R, T, 16, 1.0, True)
    plain = b.verify_logits(t.cuda().view(R, T, V), None, dev(drafts), top_k=16, want_lse=True)
    check_verify(plain, t.float().numpy(), drafts, None, None, R, T, 16, 1.0, True)


def ties(kind, M, V, g):
    if kind == "equal":
        return np.full((M, V), 1.5, np.float32)
    if kind == "ascending":
        return np.tile(np.arange(V, dtype=np.float32), (M, 1))
    if kind == "descending":
        return -np.tile(np.arange(V, dtype=np.float32), (M, 1))
    if kind == "few_values":
        return g.integers(0, 3, (M, V)).astype(np.float32)
    if kind == "one_lane":                             # all large values in one lane's tokens
        x = g.normal(0, 1, (M, V)).astype(np.float32)
        x[:, 4::256] += 50
        x[:, 5::256] += 50
        return x
    x = np.full((M, V), -np.inf, np.float32)           # "sparse": a handful above -inf
    for m in range(M):
        x[m, g.integers(0, V, m % 5)] = g.normal(0, 1)
    return x


@pytest.mark.parametrize("k", [0, 5, 16])
@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "few_values", "one_lane", "sparse"])
def test_hard_orders(b, kind, k):
    g = np.random.default_rng(3)
    for R, T, V in ((2, 3, 700), (1, 5, 3001), (1, 2, 66000)):
        x = ties(kind, R * T, V, g)
        drafts = g.integers(0, V, (R, T - 1)).astype(np.int32)
        drafts = near_drafts(x, drafts, R, T, k)
        dp, un = g.random((2, R, T - 1)).astype(np.float32)
        got = b.verify_logits(dev(x), None, dev(drafts), dev(dp), dev(un), R=R, top_k=k, temperature=0.9, want_lse=True)
        check_verify(got, x, drafts, dp, un, R, T, k, 0.9, True)


def test_empty_rows_and_infinities(b):
    V = 2500
    x = np.random.default_rng(0).normal(0, 1, (6, V)).astype(np.float32)
    x[0] = -np.inf
    x[1] = np.nan
    x[2, 100] = np.inf
    x[3, [100, 2000]] = np.inf
    x[4, 7] = np.nan
    drafts = np.array([[100], [100], [7]], np.int32)   # rows 0, 2 and 4
    dp, un = np.ones((3, 1), np.float32), np.zeros((3, 1), np.float32)
    for k in (0, 4):
        got = b.verify_logits(dev(x), None, dev(drafts), dev(dp), dev(un), R=3, top_k=k, want_lse=True)
        lmax, amax, tids, tlog, pdr, nacc, lse = got
        assert amax.tolist()[:4] == [-1, -1, 100, 100] and lmax.tolist()[:4] == [-np.inf, -np.inf, np.inf, np.inf]
        assert lse.tolist()[:4] == [-np.inf, -np.inf, np.inf, np.inf]
        assert pdr[:, 0].tolist() == [0.0, 1.0, 0.0] and nacc.tolist() == [0, 1, 0]
        if k:
            assert tids[0].tolist() == [-1] * 4 and tlog[1].tolist() == [-np.inf] * 4
            assert tids[3].tolist()[:2] == [100, 2000]
    want = lr.lse64(np.where(np.isnan(x[4]), -np.inf, x[4]), 1.0)
    assert abs(lse[4].item() - want) <= 93 * U * abs(want)


@pytest.mark.parametrize("R,T", [(1, 1), (2, 6)])
def test_empty_history_and_biases_still_count_the_drafts(b, R, T):
    V = 1100
    logits, rules, drafts = make(R, T, V, 3, history=0, bias=0, mask=None)
    drafts = drafts % 7 if T > 1 else drafts            # repeated drafts
    none = dict(rules, history=np.zeros(0, np.int32), history_offsets=np.zeros(R + 1, np.int64),
                n_prompt=np.zeros(R, np.int32), bias_ids=np.zeros(0, np.int32),
                bias_values=np.zeros(0, np.float32), bias_offsets=np.zeros(R + 1, np.int64))
    want = lr.ruled(logits, rules, drafts, R, T)
    d = dev(drafts) if T > 1 else None
    same(b.apply_logit_rules(dev(logits), device_rules(b, none), d, R=R), want)
    check_verify(b.verify_logits(dev(logits), device_rules(b, none), d, R=R, top_k=4), want, drafts, None, None, R, T,
                 4, 1.0, False)


@pytest.mark.parametrize("k", [0, 9])
@pytest.mark.parametrize("tau", [1e-42, 2e-38, 3e38])
def test_temperatures_at_the_ends(b, tau, k):
    # The scale log2(e) / tau overflows, is near the largest number, or is
    # subnormal: the best token has all of the probability, or each its share.
    R, T, V = 2, 3, 3001
    logits, rules, drafts = make(R, T, V, 17, mask=None)
    x = lr.ruled(logits, rules, drafts, R, T)
    drafts = near_drafts(x, drafts, R, T, k)
    x = lr.ruled(logits, rules, drafts, R, T)
    g = np.random.default_rng(k)
    dp, un = g.random((2, R, T - 1)).astype(np.float32)
    got = b.verify_logits(dev(logits), device_rules(b, rules), dev(drafts), dev(dp), dev(un), R=R, top_k=k,
                          temperature=tau, want_lse=True)
    if tau < 1:                                          # 1/tau times a maximum above 1 is beyond binary32 or close
        best = x.argmax(1)
        for i in range(R):
            for t in range(T - 1):
                assert got[4][i, t].item() == float(drafts[i, t] == best[i * T + t])
        assert not torch.isnan(got[6]).any()
    else:
        check_verify(got, x, drafts, dp, un, R, T, k, float(np.float32(tau)), True)


def test_no_rules_equals_verify_sampled(b):
    """The same logits, once through the head's own sampled epilogue."""
    from int4_output_head_amd import synth
    i = synth.int_exact_inputs(24, 3000, 256, seed=2)
    h = torch.from_numpy(i["hidden"]).view(torch.float16).cuda().view(6, 4, 256)
    w, s = torch.from_numpy(i["packed"]).cuda(), torch.from_numpy(i["scales"]).view(torch.float16).cuda()
    g = torch.Generator().manual_seed(0)
    d = b.verify_batch(h, w, s, torch.zeros(6, 3, dtype=torch.int32, device="cuda"))[1].view(6, 4)[:, :3].contiguous()
    dp, un = (torch.rand(6, 3, generator=g).cuda() for _ in range(2))
    for k in (0, 8):
        a = b.verify_sampled(h, w, s, d, dp, un, top_k=k, temperature=0.8, want_lse=True)
        c = b.verify_ruled(h, w, s, None, d, dp, un, top_k=k, temperature=0.8, want_lse=True)
        for name, u, v in zip(("lmax", "amax", "tids", "tlog", "p", "nacc", "lse"), a, c):
            if u is None:
                assert v is None
            elif name in ("p", "lse"):
                # the epilogue's p over the whole vocabulary is exp(l_d / tau - lse) with logits of several
                # hundred: either term is rounded to u |lse|, and lse itself carries 3 u |lse|
                rtol = 2e-5 + (6 * U * a[6].abs().max().item() if name == "p" else 0.0)
                assert torch.allclose(u, v, rtol=rtol, atol=1e-7), name
            else:
                assert torch.equal(u, v), name
    a = b.verify_batch(h, w, s, d)
    c = b.verify_ruled(h, w, s, None, d)
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1]) and torch.equal(a[2], c[5])


@pytest.mark.parametrize("R,T,V,H", [(1, 1, 500, 64), (1, 16, 5000, 256), (10, 4, 3001, 128), (20, 4, 2000, 64)])
def test_verify_ruled(b, R, T, V, H):
    from int4_output_head_amd import synth
    i = synth.int_exact_inputs(R * T, V, H, seed=V)
    h = torch.from_numpy(i["hidden"]).view(torch.float16).cuda()
    w, s = torch.from_numpy(i["packed"]).cuda(), torch.from_numpy(i["scales"]).view(torch.float16).cuda()
    _, rules, drafts = make(R, T, V, V)
    d = dev(drafts) if T > 1 else None
    r = device_rules(b, rules)
    logits = b.verify_batch(h, w, s, d, R=R, logits=True)[3]
    x = lr.ruled(logits.cpu().numpy(), rules, drafts, R, T)
    dp, un = np.random.default_rng(1).random((2, R, T - 1)).astype(np.float32)
    for k in (0, 6):
        got = b.verify_ruled(h, w, s, r, d, R=R, top_k=k, want_lse=True)
        check_verify(got, x, drafts, None, None, R, T, k, 1.0, True)
        if T > 1:
            got = b.verify_ruled(h, w, s, r, d, dev(dp), dev(un), R=R, top_k=k, temperature=1.4)
            check_verify(got, x, drafts, dp, un, R, T, k, 1.4, False)
    ws = b.Workspace(b.load_library().verify_lm_head_int4_ruled_workspace_bytes(R, T, V, H, 6), h.device)
    for _ in range(2):
        again = b.verify_ruled(h, w, s, r, d, R=R, top_k=6, want_lse=True, workspace=ws)
        first = b.verify_ruled(h, w, s, r, d, R=R, top_k=6, want_lse=True)
        for u, v in zip(again, first):
            assert u is None or torch.equal(u, v)


def test_streams_and_graphs(b):
    """Two captured graphs, the eager calls between their replays, and two
    streams at once, on changing logits, histories and drafts."""
    from int4_output_head_amd import synth
    R, T, V, H = 3, 4, 5000, 64
    logits, rules, drafts = make(R, T, V, 9)
    r, x, d = device_rules(b, rules), dev(logits), dev(drafts)
    history = r.tensors[0]
    i = synth.int_exact_inputs(R * T, V, H, seed=1)
    h = torch.from_numpy(i["hidden"]).view(torch.float16).cuda()
    w, s = torch.from_numpy(i["packed"]).cuda(), torch.from_numpy(i["scales"]).view(torch.float16).cuda()

    def run():
        return [b.apply_logit_rules(x, r, d, R=R)] + \
            [t for t in b.verify_logits(x, r, d, R=R, top_k=8, want_lse=True) if t is not None] + \
            [t for t in b.verify_ruled(h, w, s, r, d, R=R, top_k=8, want_lse=True) if t is not None]
    run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run()
        graphs.append((g, out))
    gen = torch.Generator().manual_seed(0)
    for _ in range(4):
        x.copy_(torch.randn(x.shape, generator=gen) * 3)
        history.copy_(torch.randint(0, V, history.shape, generator=gen, dtype=torch.int32))
        d.copy_(torch.randint(0, V, d.shape, generator=gen, dtype=torch.int32))
        want = run()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for u, v in zip(out, want):
                assert torch.equal(u, v)
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        with torch.cuda.stream(st):
            outs.append(run())
    torch.cuda.synchronize()
    for out in outs:
        for u, v in zip(out, want):
            assert torch.equal(u, v)


def test_refusals(b):
    logits, rules, drafts = make(2, 3, 100, 1)
    x, r, d = dev(logits), device_rules(b, rules), dev(drafts)
    kw = {k: None if v is None else torch.from_numpy(v.view(np.int32) if k == "mask" else v).cuda()
          for k, v in rules.items()}
    for change in (dict(history=None), dict(history_offsets=None), dict(repetition=torch.ones(3, device="cuda")),
                   dict(bias_values=None), dict(bias_ids=kw["bias_ids"][:-1]), dict(mask=None),
                   dict(n_prompt=kw["n_prompt"][:1])):
        with pytest.raises(ValueError):
            b.LogitRules(**{**kw, **change})
    for change in (dict(history=kw["history"].long()), dict(mask=kw["mask"].long()), dict(mask=kw["mask"][0]),
                   dict(presence=kw["presence"].half()), dict(repetition=kw["repetition"].cpu())):
        with pytest.raises(TypeError):
            b.LogitRules(**{**kw, **change})
    few = b.LogitRules(**{**kw, "mask_index": kw["mask_index"][:4]})
    short = b.LogitRules(mask=torch.zeros(6, 3, dtype=torch.int32, device="cuda"))
    u = torch.zeros(2, 2, device="cuda")
    for bad in (lambda: b.apply_logit_rules(x, r, d), lambda: b.apply_logit_rules(x, r, d, R=4),
                lambda: b.apply_logit_rules(x, r, None, R=2), lambda: b.apply_logit_rules(x, r, d[:1], R=2),
                lambda: b.apply_logit_rules(x, r, d, R=3), lambda: b.apply_logit_rules(x, few, d, R=2),
                lambda: b.apply_logit_rules(x, short, d, R=2), lambda: b.apply_logit_rules(x, r, d, R=2, out=x[:5]),
                lambda: b.verify_logits(x, r, d, u, None, R=2), lambda: b.verify_logits(x.t(), r, d, R=2),
                lambda: b.verify_logits(x[:0], None, R=1)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: b.verify_logits(x, r, d, R=2, top_k=17), lambda: b.verify_logits(x, r, d, R=2, temperature=0.0),
                lambda: b.verify_logits(x[:, :4], None, d, R=2, top_k=5)):
        with pytest.raises(RuntimeError):
            bad()
