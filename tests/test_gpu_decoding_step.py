"""The operators around the head in the order of a decoding step: calibrated
weights, the 8-bit norm, a linear layer onto the residual stream, the final
norm, and the head's verification under rules -- against the plain forms, each
fed with the GPU's own output of the step before it."""
import numpy as np
import pytest
import torch

from oracle import logit_rules as lr
from oracle import rows

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("R,T,dt", [(1, 1, torch.float16), (1, 16, torch.bfloat16), (6, 4, torch.float16),
                                    (20, 4, torch.bfloat16)])
def test_decoding_step(R, T, dt):
    from int4_output_head_amd import binding as b
    M, H, V = R * T, 512, 3001
    g = torch.Generator().manual_seed(M)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    # one calibration for the layer and one for the head (the library's own offline step)
    acts = (2 * rnd(300, H)).to(torch.float16).cuda()
    layer, layer_scales, _ = b.requantize((0.5 * rnd(H, H)).to(torch.float16).cuda(), acts)
    head, head_scales, _ = b.requantize((0.5 * rnd(V, H)).to(torch.float16).cuda(), acts)
    x, stream = rnd(M, H).to(dt).cuda(), (2 * rnd(M, H)).to(dt).cuda()
    w1, w2 = (1 + 0.2 * rnd(2, H)).to(dt).cuda()
    bias = (0.1 * rnd(H)).to(dt).cuda()

    codes, row_scales, stream1 = b.rms_norm_int8(x, w1, stream, channel_scales=layer_scales)
    y = b.linear_int4(codes, row_scales, layer, bias=bias, activation="silu", out_dtype=dt)
    hidden, stream2 = b.rms_norm(y, w2, stream1)
    assert hidden.dtype == torch.float16
    drafts = torch.randint(0, V, (R, T - 1), generator=g, dtype=torch.int32).cuda() if T > 1 else None
    rules = dict(lr.NONE, history=torch.randint(0, V, (R * 20,), generator=g, dtype=torch.int32).numpy(),
                 history_offsets=20 * np.arange(R + 1), n_prompt=np.full(R, 8, np.int32),
                 repetition=np.full(R, 1.2, np.float32), presence=np.full(R, 0.3, np.float32))
    r = b.LogitRules(**{k: None if v is None else torch.from_numpy(v).cuda() for k, v in rules.items()})
    got = b.verify_ruled(hidden, head, head_scales, r, drafts, R=R, top_k=5, want_lse=True)

    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    assert np.array_equal(codes.cpu().numpy(), rows.codes32(x.float().cpu().numpy(), w1.float().cpu().numpy(),
                                                            stream.float().cpu().numpy(),
                                                            layer_scales.float().cpu().numpy()))
    z, pre, s = rows.linear64(codes.cpu().numpy(), f(row_scales), layer.cpu().numpy(), None, f(bias), "silu")
    tol = 12 * U * (np.abs(s) + np.abs(pre)) + torch.finfo(dt).eps / 2 * np.abs(z) + 2.0 ** -25
    assert np.all(np.abs(f(y) - z) <= tol * 1.001)
    want = rows.norm64(f(y), f(w2), f(stream1), 1e-6)
    assert np.all(np.abs(f(hidden) - want) <= np.abs(want) * (2.0 ** -11 + 33 * U) + 2.0 ** -25)
    assert torch.equal(stream2, (y.float() + stream1.float()).to(dt))
    d = drafts.cpu().numpy() if T > 1 else np.zeros((R, 0), np.int32)
    logits = b.verify_batch(hidden, head, head_scales, drafts, R=R, logits=True)[3]
    ruled = lr.ruled(logits.cpu().numpy(), rules, d, R, T)
    for m in range(M):
        ids, val = lr.top(ruled[m], 5)
        assert got[2][m].tolist() == ids.tolist() and got[3][m].tolist() == val.tolist()
    n = [next((t for t in range(T - 1) if got[1][i * T + t] != d[i, t]), T - 1) for i in range(R)]
    assert got[5].tolist() == n
