"""The largest number of rows that the quantisation to 4 bits takes (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_quantize_2_31_rows():
    """2^31 - 1 rows of 32 channels, more than go as one long row: a workgroup walks 32769 of them, and its step
    past the last one passes 31 bits."""
    from int4_output_head_amd import binding as b
    M, H = (1 << 31) - 1, 32
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 185 * 10 ** 9:
        pytest.skip("needs 174 GB of GPU memory")
    x = torch.empty(M, H, dtype=torch.float16, device="cuda").fill_(2.5)
    n = 70000                                   # more than the rows a step apart
    ends = [(0, n), (M // 2, n), (M - n, n)]
    parts = [torch.randn(n, H, generator=torch.Generator().manual_seed(i)).half().cuda() for i in range(3)]
    for (at, k), part in zip(ends, parts):
        x[at: at + k] = part
    codes, scales = b.quantize_mxfp4(x)
    torch.cuda.synchronize()
    for (at, k), part in zip(ends, parts):
        c, s = b.quantize_mxfp4(part)
        assert torch.equal(codes[at: at + k], c) and torch.equal(scales[at: at + k], s)
    # 2.5 = 5 * 2^-1: a tie between 4 and 6, which goes to the even code, 4 (6)
    for at in (n, M // 2 - 1, M // 2 + n, M - n - 1):
        assert (codes[at] == 0x66).all() and scales[at].item() == 126
    del x, codes, scales
    torch.cuda.empty_cache()
