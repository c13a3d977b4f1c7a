"""Gates whose sigmoid is below the normal numbers of binary32, on rows large enough
to show it (GPU).

The sigmoid is off by 6 half steps at most, which are 2^-24 of a normal value and 2^-150
of a subnormal one; the product and the sum round once each."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def b():
    from int4_output_head_amd import binding
    return binding


def close(total, x, gate, residual, scale=1.0):
    x, gate, residual, total = (t.double().cpu().numpy() for t in (x, gate, residual, total))
    s = np.exp(-np.logaddexp(0.0, -gate))
    want = residual + x * s * scale
    off = (6 * np.maximum(2.0 ** -24 * s, 2.0 ** -150) * np.abs(x * scale)
           + 3 * 2.0 ** -24 * (np.abs(want) + np.abs(x * s * scale)))
    assert np.all(np.abs(total - want) <= off + 2.0 ** -149), float(np.max(np.abs(total - want) / off))


@pytest.mark.parametrize("size", [1e20, 1e30, 3e37])
@pytest.mark.parametrize("rows", [False, True])
def test_far_below(b, size, rows):
    gate = torch.cat([torch.linspace(-105, -80, 5000), torch.tensor([-87.33, -87.34, -87.0, -86.9, -103.9, -104.1, -90.0])])
    H = len(gate)
    g = torch.Generator().manual_seed(1)
    x = size * (1.0 + torch.rand(3, H, generator=g))
    residual = torch.zeros(3, H)
    z = gate.expand(3, H).contiguous() if rows else gate
    total = b.rms_norm_block(x.cuda(), residual.cuda(), gate=z.cuda(), gate_activation="sigmoid")[1]
    close(total, x, gate.expand(3, H), residual)
    assert (total[:, gate > -103].cpu() > 0).all()


def test_beside_ordinary_ones(b):
    """One gate in a row that is far below changes no other one's bits, whether it lies in the same lane, the same
    wave or another."""
    H = 2048
    g = torch.Generator().manual_seed(2)
    x, residual = torch.randn(4, H, generator=g).cuda(), torch.randn(4, H, generator=g).cuda()
    gate = 8.0 * torch.randn(4, H, generator=g).cuda()
    want = b.rms_norm_block(x, residual, gate=gate, gate_activation="sigmoid")[1]
    for at in (0, 7, 100, 1000, 2047):
        one = gate.clone()
        one[:, at] = -95.0
        total = b.rms_norm_block(x, residual, gate=one, gate_activation="sigmoid")[1]
        keep = torch.arange(H, device="cuda") != at
        assert torch.equal(total[:, keep], want[:, keep]) and torch.equal(total[:, at], residual[:, at])


def test_bfloat16_rows(b):
    H = 264
    x = torch.full((2, H), 1e30, dtype=torch.bfloat16)
    gate = torch.linspace(-100, -88, H).to(torch.bfloat16)
    total = b.rms_norm_block(x.cuda(), torch.zeros_like(x).cuda(), gate=gate.cuda(), gate_activation="sigmoid")[1]
    s = np.exp(-np.logaddexp(0.0, -gate.double().numpy()))
    want = x.double().numpy() * s
    off = 6 * 2.0 ** -150 * x.double().numpy() + want * (2.0 ** -9 + 2.0 ** -23) * 2
    assert np.all(np.abs(total.double().cpu().numpy() - want) <= off)


def test_ends_and_nan(b):
    gate = torch.tensor([-104.5, -1e30, -float("inf"), float("nan"), 104.5, 1e30, float("inf"), -88.0] * 8)
    x, residual = torch.full((2, 64), 1e30), torch.zeros(2, 64)
    total = b.rms_norm_block(x.cuda(), residual.cuda(), gate=gate.cuda(), gate_activation="sigmoid")[1].cpu().view(2, 8, 8)
    assert (total[..., :3] == 0).all() and total[..., 3].isnan().all() and (total[..., 4:7] == x[0, 0]).all()
    assert (total[..., 7] > 6e-9).all() and (total[..., 7] < 6.1e-9).all()   # 1e30 exp(-88) = 6.05e-9
