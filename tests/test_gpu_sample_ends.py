"""Unfiltered draws at the ends of the uniform numbers' range, in rows whose ends
lie far below the best token (GPU).

A chunk of 1024 tokens is drawn by its sum, in units of 2^-44 (151936 tokens), of
which its tokens may each have less than half: 31.6 temperatures below the best a
mass is 0.33 units, and 1024 of them 336."""
import math

import numpy as np
import pytest
import torch

from oracle import logit_rules as lr
from oracle import sampling
from tests.test_gpu_sample import check

pytestmark = pytest.mark.gpu
UNIFORM = [0.0, -1.0, 2.0 ** -40, 2.0 ** -37, 2.0 ** -32, 0.5, 1 - 2.0 ** -24, 1.0, 7.0]
FAR = 31.6
PLAIN = (1.0, 0, 1.0, 0.0)


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def far_ends(V, temperature, first=4096, n=1024):
    """`first` tokens at -infinity, n at FAR temperatures below the best, which lies
    at 3/4; the last n likewise; between them nothing that weighs."""
    x = torch.full((V,), -500.0 * temperature)
    x[:first] = -math.inf
    x[first: first + n] = -FAR * temperature
    x[V - n:] = -FAR * temperature
    x[3 * V // 4] = 0.0
    return x


@pytest.mark.parametrize("V", [9000, 151936, 1300000])
@pytest.mark.parametrize("temperature", [1.0, 0.25, 4.0])
def test_far_chunks(b, V, temperature):
    x = far_ends(V, temperature)
    M = len(UNIFORM)
    u = torch.tensor(UNIFORM)
    rows = x.expand(M, V).contiguous()
    got = b.sample_logits(rows.cuda(), u.cuda(), R=M, temperature=temperature)
    ids = got[0].tolist()
    s = (temperature, 0, 1.0, 0.0)
    check(got, rows.double().numpy(), [s] * M, u)
    assert ids[0] == ids[1] == 4096 and ids[4:7] == [3 * V // 4] * 3 and ids[7] == ids[8] == V - 1
    # Within the far chunk tokens keep their share: the target is rounded down by up to a unit, and the chunk's sum by
    # up to half of one.
    bits = 62 - (V - 1).bit_length()
    tokens_a_unit = 2.0 ** -bits / math.exp(-FAR)
    tokens = sampling.kept(rows[0].double().numpy(), *s)
    for i in (2, 3):
        want = sampling.draw(rows[0].double().numpy(), tokens, temperature, UNIFORM[i])[0]
        assert 4096 <= ids[i] < 5120 and abs(ids[i] - want) <= 1.5 * tokens_a_unit + 1


@pytest.mark.parametrize("V", [20000, 151936])
def test_far_chunks_under_a_mask(b, V):
    """Refused tokens are none of the drawn ones, whatever lies there."""
    x = far_ends(V, 1.0)
    x[:4096] = 3.0                              # likely, but refused
    M = len(UNIFORM)
    words = np.full((1, (V + 31) // 32), 0xFFFFFFFF, np.uint32)
    words[0, :128] = 0
    rules = dict(lr.NONE, mask=words, mask_index=np.zeros(M, np.int32))
    dev = b.LogitRules(mask=torch.from_numpy(words.view(np.int32)).cuda(),
                       mask_index=torch.zeros(M, dtype=torch.int32).cuda())
    rows = x.expand(M, V).contiguous()
    u = torch.tensor(UNIFORM)
    got = b.sample_logits(rows.cuda(), u.cuda(), dev, R=M)
    check(got, lr.ruled(rows.numpy(), rules, np.zeros((M, 0), np.int32), M, 1).astype(np.float64), [PLAIN] * M, u)
    ids = got[0].tolist()
    assert min(ids) == ids[0] == ids[1] == 4096 and ids[7] == ids[8] == V - 1


def test_a_chunk_of_tokens_below_half_a_unit(b):
    """Two chunks, units of 2^-50: the first chunk's tokens have 0.3 of them each."""
    V = 2048
    x = torch.full((V,), -math.inf)
    x[:1024] = math.log(0.3) - 50 * math.log(2.0)
    x[1500] = 0.0
    M = len(UNIFORM)
    rows = x.expand(M, V).contiguous()
    u = torch.tensor(UNIFORM)
    got = b.sample_logits(rows.cuda(), u.cuda(), R=M)
    check(got, rows.double().numpy(), [PLAIN] * M, u)
    assert got[0].tolist() == [0, 0] + [1500] * 7
    assert abs(got[1][0].item() / (0.3 * 2.0 ** -50) - 1) < 2.0 ** -18   # the logit's own rounding: 2^-19 of a mass


@pytest.mark.parametrize("seed", range(4))
def test_ordinary_logits_with_one_far_above(b, seed):
    V = 151936
    x = 2.0 * torch.randn(V, generator=torch.Generator().manual_seed(seed))
    x[V // 3] = 22.0
    M = len(UNIFORM)
    rows = x.expand(M, V).contiguous()
    u = torch.tensor(UNIFORM)
    got = b.sample_logits(rows.cuda(), u.cuda(), R=M, temperature=0.5)
    inside = [0, 2, 3, 4, 5, 6]                 # (from 1 on the 64-bit form draws by 1 - 2^-53, within the far end)
    check([None if t is None else t[inside] for t in got], rows[inside].double().numpy(), [(0.5, 0, 1.0, 0.0)] * 6,
          u[inside])
    ids, want = got[0].tolist(), [sampling.draw(rows[0].double().numpy(), np.arange(V), 0.5, v)[0] for v in UNIFORM]
    # (a chunk that sums up to less than half a unit is none)
    assert ids[0] == ids[1] and ids[0] < 2048 and ids[4:7] == want[4:7] and ids[7] == ids[8] and ids[7] >= V - 2048


@pytest.mark.parametrize("V", [9000, 151936])
def test_a_draft_set_apart(b, V):
    """What remains beside the draft is drawn likewise: the draft is 40 above the row's other tokens."""
    x = far_ends(V, 1.0)
    d = V // 2
    x[d] = 40.0
    M = len(UNIFORM)
    rows = x.expand(2 * M, V).contiguous()
    u = torch.tensor(UNIFORM).repeat_interleave(2)
    drafts = torch.full((M, 1), d, dtype=torch.int32)
    accept = torch.full((M, 1), 0.5)
    got = b.sample_logits(rows.cuda(), u.cuda(), None, drafts.cuda(), R=M, accept=accept.cuda())
    # the rows behind the drafts hold the draft's token still, beside which the far ones, 1024 e^-71.6 = 2^-93 of it,
    # are below half a unit (2^-45); numbers below 0 count as 0, to which the 64-bit form allows what is near
    check(got, rows.double().numpy(), [PLAIN] * M, u.clamp(min=0), drafts, accept, M, 2)
    ids = got[0].view(M, 2)[:, 0].tolist()
    assert ids[0] == ids[1] == 4096 and ids[4:7] == [3 * V // 4] * 3 and ids[7] == ids[8] == V - 1
