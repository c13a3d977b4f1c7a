"""Thousands of candidates under top_k and top_p, which the draw moves within the
row's place to have fewer of them: once, twice, or not where there is no room
(GPU).  What lies behind the workspace stays as it is, and so do the rows beside
each other."""
import pytest
import torch

from oracle import sampling
from tests.test_gpu_sample import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def shelf(V, far, seed):
    """Logits uniform over [0, 4); a token in 64 at -1, which holds the bound of top_k
    down so that the shelf is above it; `far` or nearly as many at -30."""
    x = 4.0 * torch.rand(V, generator=torch.Generator().manual_seed(seed))
    v = torch.arange(V)
    x[(v * 7919) % V < far] = -30.0
    x[::64] = -1.0
    return x


# (V, tokens far down, settings): with n candidates of V, m of them down to top_k's
# border and l down to top_p's, the second move has room where n + m + l <= V (numbers to within some tens).
CASES = [(151936, 12000, (1.0, 9000, 0.999, 0.0)),     # 140100, 9200, 9000: room for the first move alone
         (151936, 12000, (1.0, 9000, 0.9999, 0.0)),
         (100000, 7500, (1.0, 6000, 0.999, 0.0)),      # 92600, 6050, 6050: likewise
         (300000, 11000, (2.0, 9000, 0.99, 0.0)),      # 289200, 9300, 8900: likewise
         (151936, 90000, (1.0, 9000, 0.999, 0.0)),     # 63300, 9100, 9100: room for both
         (151936, 7000, (1.0, 9000, 0.3, 0.0)),        # 145000, 9100, 2600: room for the second alone
         (151936, 12000, (1.0, 9000, 0.999, 0.05))]


@pytest.mark.parametrize("V,far,s", CASES)
def test_candidates_move_within_their_row(b, V, far, s):
    M = 4
    x = torch.stack([shelf(V, far, V + i) for i in range(M)])
    u = torch.tensor([0.0, 0.31, 0.77, 1 - 2.0 ** -24])
    L, dev, du = b.load_library(), x.cuda(), u.cuda()
    need = L.sample_logits_workspace_bytes(M, 1, V)
    ids, probs = torch.empty(M, dtype=torch.int32).cuda(), torch.empty(M).cuda()
    ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8).cuda()
    st = L.sample_logits_rows(dev.data_ptr(), V, 2, None, M, 1, V, None, b._SAMPLING.pack(0, 0, 0, 0, *s),
                              du.data_ptr(), None, ids.data_ptr(), probs.data_ptr(), None, None, ws.data_ptr(), need,
                              torch.cuda.current_stream().cuda_stream)
    assert st == 0
    check((ids, probs, None, None), x.double().numpy(), [s] * M, u)
    assert bool((ws[need:] == 0xA5).all())


@pytest.mark.parametrize("V,far,s", CASES[:2] + CASES[4:6])
def test_with_drafts(b, V, far, s):
    R, T = 2, 3
    x = torch.stack([shelf(V, far, V + i) for i in range(R * T)])
    g = torch.Generator().manual_seed(V)
    u, accept = torch.rand(R * T, generator=g), torch.rand(R, T - 1, generator=g)
    best = x.topk(2, dim=1).indices.view(R, T, 2)
    d = torch.stack((best[:, 0, 0], best[:, 1, 1]), dim=1).to(torch.int32).contiguous()
    got = b.sample_logits(x.cuda(), u.cuda(), None, d.cuda(), R=R, temperature=s[0], top_k=s[1], top_p=s[2],
                          min_p=s[3], accept=accept.cuda())
    check(got, x.double().numpy(), [s] * R, u, d, accept, R, T)


def test_a_row_alone_gives_the_bits_of_the_batch(b):
    V, far, s = CASES[0]
    x = torch.stack([shelf(V, far, i) for i in range(24)]).cuda()
    u = torch.rand(24, generator=torch.Generator().manual_seed(1)).cuda()
    kw = dict(temperature=s[0], top_k=s[1], top_p=s[2])
    ids, probs, _, _ = b.sample_logits(x, u, R=24, **kw)
    for m in (0, 7, 22, 23):
        one = b.sample_logits(x[m:m + 1], u[m:m + 1], R=1, **kw)
        assert torch.equal(one[0][0], ids[m]) and torch.equal(one[1][0], probs[m])
        assert int(ids[m]) in sampling.kept(x[m].double().cpu().numpy(), *s)
