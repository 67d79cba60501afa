"""GPU tests of the block-FP8 feed-forward operators on values of very
different size: what one part of a sum holds must not cost another its bits."""
import pytest
import torch

import int8_gemm_gemv_b200 as bsq
from test_gpu_block_ffn import Moe

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert bsq.debug_take_timeouts() == 0


@pytest.mark.parametrize("rise", [2.0**27, 2.0**60])
@pytest.mark.parametrize("t,h,i", [(3, 512, 384), (12, 256, 1408)])
def test_moe_act_of_one_block_far_above_the_others(t, h, i, rise):
    """K block 1 of act rises by a power of two.  The first 128 outputs have no
    down weight there, so none of their bits may change."""
    m = Moe(t, h, i, 4, 2, 1, seed=31)
    m.s2[:, 0, 1] = 0
    m()
    m.check("level")
    level = m.out[:t, :128].clone()
    m.s13[:, i // 128 + 1] *= rise  # the up rows of that block
    m.out.view(torch.uint8).fill_(0xFF)
    m()
    m.check("raised")
    assert torch.equal(m.out[:t, :128].view(torch.int16), level.view(torch.int16))
    assert (m.out[:t, :128] != 0).any() and (m.out[:t, 128:].abs().amax() > 2**20 * level.abs().amax())


@pytest.mark.parametrize("group", [0, 3, 7])
def test_moe_act_of_sixteen_rows_far_below_their_block(group):
    """Sixteen values of act about 2^-27 of their block's largest, and down
    weights for those alone: kept to 2^-38 of that largest."""
    t, h, i, e = 3, 256, 256, 2
    m = Moe(t, h, i, e, 2, 1, seed=33)
    rows = slice(128 + 16 * group, 128 + 16 * group + 16)
    tiny = torch.where(torch.arange(h, device="cuda") % 2 == 0, 0x08, 0x88).to(torch.uint8)  # +-2^-6
    m.w13[:, rows] = tiny  # gate
    m.w13[:, i + rows.start:i + rows.stop] = tiny
    keep = m.w2[:, :, rows].clone()
    m.w2[:] = 0
    m.w2[:, :, rows] = keep
    m()
    m.check(group)
    assert (m.out[:t] != 0).float().mean() > 0.9
