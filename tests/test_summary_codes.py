"""int8 codes where their scale is subnormal.

fl(max / 127) is a multiple of 2^-149 there, so the largest values can be more than
127 scales: their codes are held to 127 and keep their sign.
"""
import numpy as np
import pytest
import torch

from test_tree import kvq, make  # noqa: F401 (fixture)

TINY = 2.0 ** -149


def clamped_codes(x, scale):
    y = np.rint(x / np.where(scale > 0, scale, np.float32(1)))
    return np.where(scale > 0, np.clip(y, -127, 127), 0).astype(np.int8)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 256])
@pytest.mark.parametrize("unit", [1, 27, 18, 100])
def test_summary_of_subnormal_scales(kvq, d, unit):  # noqa: F811
    c = make(kvq, 1, 2, 128, d, 0)
    code = torch.tensor([[7, -7, 1, -3, 6, -5, 0, 2] * (d // 8)], device="cuda").expand(32, d)
    packed = ((code[:, 0::2] + 8) | (code[:, 1::2] + 8) << 4).to(torch.uint8)
    c.k_codes.copy_(packed)
    c.k_scales.fill_(unit * TINY)
    assert float(c.k_scales[0, 0, 0, 0]) > 0  # (a subnormal survives)
    for block in (32, 64, 128):
        s = kvq.BlockSummary(c, block).update()
        # every token of a block is the same: the mean key is code * scale, exactly
        mean = code[0].cpu().numpy().astype(np.float32) * np.float32(unit * TINY)
        scale = np.abs(mean).max() / np.float32(127)
        want = clamped_codes(mean, scale)
        assert bool((s.scales == float(scale)).all())
        assert np.array_equal(s.codes.cpu().numpy(), np.broadcast_to(want, s.codes.shape))


@pytest.mark.gpu
@pytest.mark.parametrize("d,blocks", [(64, 24), (128, 24), (128, 2000)])
def test_choice_with_a_subnormal_query_row(kvq, d, blocks):  # noqa: F811
    # q = 190 tiny in feature 0, 3 tiny in feature 1: scale 1 tiny, codes 127 and 3. Block 5
    # alone has a positive mean in feature 0, block 9 the largest in feature 1, the others are
    # negative in feature 0. Scores are s_q * s_b * dot, about 1e-45 * 8e33 * 127^2.
    c = make(kvq, 1, 1, 32 * blocks, d, 0)
    code = torch.zeros((blocks, 32, d), dtype=torch.int64, device="cuda")
    code[:, :, 0] = -7
    code[5, :, 0] = 7
    code[9, :, 0] = 0
    code[9, :, 1] = 7
    c.k_codes.copy_(((code[..., 0::2] + 8) | (code[..., 1::2] + 8) << 4).to(torch.uint8))
    c.k_scales.fill_(1e35)
    s = kvq.BlockSummary(c, 32).update()
    q = torch.zeros((1, 1, 1, d), device="cuda")
    q[..., 0], q[..., 1] = 190 * TINY, 3 * TINY
    a = kvq.AttendBlocks(c, q, s, 1, out_dtype="f32")
    a.run()
    assert a.selected.flatten().tolist() == [5]
