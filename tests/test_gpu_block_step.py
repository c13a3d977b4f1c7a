"""The norms around a block, its linear layers in 4-bit floating point and the
sampler run together, as a model's decoding step calls them: each operator's
output against its oracle on the operand that it was given, and the captured
step against the eager one (GPU)."""
import numpy as np
import pytest
import torch

from oracle import logit_rules as lr
from oracle import mxfp4
from tests.test_gpu_block_norm import close
from tests.test_gpu_mxfp4 import check as check_linear
from tests.test_gpu_sample import check as check_sample

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


class Step:
    """A gated block's output onto the residual stream, a feed-forward layer, the
    final norm, a head and a token for each row."""

    def __init__(self, b, R, T, H, F, V, dt, seed):
        self.b, self.R, self.T, self.V, self.dt = b, R, T, V, dt
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        M = R * T
        self.x, self.residual, self.gate = (rnd(M, H).to(dt).cuda() for _ in range(3))
        self.post, self.pre, self.last = ((1 + 0.2 * rnd(H)).to(dt).cuda() for _ in range(3))
        self.up = b.quantize_mxfp4((0.05 * rnd(F, H)).cuda())
        self.down = b.quantize_mxfp4((0.05 * rnd(H, F)).cuda())
        self.head = b.quantize_mxfp4((0.2 * rnd(V, H)).cuda())
        self.bias = (0.1 * rnd(F)).to(dt).cuda()
        self.uniforms, self.accept = torch.rand(M, generator=g).cuda(), torch.rand(R, T - 1, generator=g).cuda()
        self.drafts = torch.randint(0, V, (R, T - 1), generator=g).to(torch.int32).cuda()
        n = 12
        self.rules = dict(lr.NONE, history=torch.randint(0, V, (n * R,), generator=g).to(torch.int32).numpy(),
                          history_offsets=n * np.arange(R + 1), n_prompt=np.full(R, n // 2, np.int32),
                          repetition=np.full(R, 1.2, np.float32), presence=np.full(R, 0.3, np.float32))
        self.device_rules = b.LogitRules(**{k: torch.from_numpy(v).cuda() for k, v in self.rules.items()
                                            if v is not None})

    def run(self):
        b, k = self.b, {}
        k["y"], k["h"] = b.rms_norm_block(self.x, self.residual, self.post, self.pre, gate=self.gate,
                                          gate_activation="sigmoid", scale=0.5, out_dtype=self.dt)
        k["qy"] = b.quantize_mxfp4(k["y"])
        k["f"] = b.linear_mxfp4(*k["qy"], *self.up, bias=self.bias, activation="silu", out_dtype=self.dt)
        k["qf"] = b.quantize_mxfp4(k["f"])
        k["o"] = b.linear_mxfp4(*k["qf"], *self.down, residual=k["h"], out_dtype=self.dt)
        k["z"], k["sum"] = b.rms_norm_block(k["o"], k["h"], None, self.last, out_dtype=self.dt)
        k["qz"] = b.quantize_mxfp4(k["z"])
        k["logits"] = b.linear_mxfp4(*k["qz"], *self.head, out_dtype=torch.float32)
        k["sample"] = b.sample_logits(k["logits"], self.uniforms, self.device_rules, self.drafts, R=self.R,
                                      temperature=0.9, top_k=40, top_p=0.95, accept=self.accept)
        return k


def host(pair):
    return tuple(t.cpu() for t in pair)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("R,T,H,F,V", [(1, 4, 256, 640, 1500), (9, 3, 512, 1056, 2048), (40, 4, 1024, 2080, 5000)])
def test_every_operator_on_its_operand(b, R, T, H, F, V, dt):
    s = Step(b, R, T, H, F, V, dt, H + F)
    k = s.run()
    close((k["y"], k["h"]), dict(x=s.x, residual=s.residual, post_weight=s.post, pre_weight=s.pre, gate=s.gate),
          "sigmoid", 0.5)
    for rows, codes in (("y", "qy"), ("f", "qf"), ("z", "qz")):
        want = mxfp4.quantize(k[rows].double().cpu().numpy())
        for got, w in zip(host(k[codes]), want):
            assert np.array_equal(got.numpy(), w)
    check_linear(k["f"], (*host(k["qy"]), *host(s.up)), "silu", s.bias.cpu())
    check_linear(k["o"], (*host(k["qf"]), *host(s.down)), None, None, k["h"].cpu())
    close((k["z"], k["sum"]), dict(x=k["o"], residual=k["h"], post_weight=None, pre_weight=s.last, gate=None))
    check_linear(k["logits"], (*host(k["qz"]), *host(s.head)))
    ruled = lr.ruled(k["logits"].cpu().numpy(), s.rules, s.drafts.cpu().numpy(), R, T)
    check_sample(k["sample"], ruled.astype(np.float64), [(0.9, 40, 0.95, 0.0)] * R, s.uniforms, s.drafts.cpu(),
                 s.accept.cpu(), R, T)


def same(a, b):
    for name in a:
        for x, y in zip(*((v,) if isinstance(v, torch.Tensor) else v for v in (a[name], b[name]))):
            assert torch.equal(x, y), name


@pytest.mark.parametrize("R,T", [(1, 4), (40, 4)])
def test_two_captured_steps(b, R, T):
    """Two graphs of steps with operands of their own, replayed in turn and on a second stream."""
    steps = [Step(b, R, T, 512, 1056, 3001, torch.bfloat16, seed) for seed in (1, 2)]
    for s in steps:
        s.run()
    torch.cuda.synchronize()
    graphs, got = [], []
    for s in steps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(s.run())
    side = torch.cuda.Stream()
    for i in range(3):
        for s in steps:
            s.x.copy_(s.x.roll(1 + i, dims=1))
            s.uniforms.copy_(torch.rand_like(s.uniforms))
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for s, g in zip(steps, got):
            same(s.run(), g)
            torch.cuda.synchronize()


def test_rows_of_a_longer_batch(b):
    """Rows do not depend on the others beside them: quantisation and norms to the bit."""
    s = Step(b, 8, 2, 512, 544, 1000, torch.float16, 5)
    y, h = b.rms_norm_block(s.x, s.residual, s.post, s.pre, gate=s.gate)
    for r in (0, 7, 15):
        one = slice(r, r + 1)
        y1, h1 = b.rms_norm_block(s.x[one], s.residual[one], s.post, s.pre, gate=s.gate[one])
        assert torch.equal(y1, y[one]) and torch.equal(h1, h[one])
        for a, w in zip(b.quantize_mxfp4(y1), b.quantize_mxfp4(y)):
            assert torch.equal(a, w[one])
