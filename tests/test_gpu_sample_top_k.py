"""top_k around the numbers at which its bound is taken from more tokens of each chunk,
and past those that it reaches (GPU)."""
import pytest
import torch

from tests.test_gpu_sample import check, logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


@pytest.mark.parametrize("V,ks", [(600000, (256, 257, 293, 294, 512, 513, 1024, 1025)), (270000, (132, 133, 257, 264, 265)),
                                  ((1 << 20) + 5, (256, 257, 512, 513)), (151936, (9536, 9537)), (300000, (16384, 16385))])
def test_around_its_steps(b, V, ks):
    x = logits(2, V, torch.float32, V, spread=3.0)
    u = torch.tensor([0.41, 1 - 2.0 ** -24])
    for k in ks:
        for s in ((1.0, k, 1.0, 0.0), (3.0, k, 0.97, 0.0)):
            got = b.sample_logits(x.cuda(), u.cuda(), R=2, temperature=s[0], top_k=s[1], top_p=s[2], min_p=s[3])
            check(got, x.double().numpy(), [s] * 2, u)
