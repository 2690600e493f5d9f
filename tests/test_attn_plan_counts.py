"""The forward's split counts and the order of its blocks at sizes whose times the plan's rule was measured at (152 SMs)."""
import pytest

import attention_kl_divergence_streamkl_gb300 as skl
from attention_kl_divergence_streamkl_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


@pytest.mark.parametrize("B,H,HK,NQ,NK,D,splits", [
    (1, 8, 8, 1, 4096, 128, 16),    # two key tiles a block in one wave of 128 blocks; 32 would be two waves
    (1, 4, 4, 1, 4096, 128, 32),    # a key tile a block
    (1, 8, 8, 1, 512, 128, 4),
    (1, 8, 8, 1, 256, 128, 1),      # two tiles: a second launch costs more than it saves
    (1, 8, 8, 512, 512, 128, 1),    # the partials of 4096 rows cost more than the splits save: 11.7 us, 15.2 with four
    (1, 32, 8, 16384, 16384, 128, 1),
])
def test_split_counts(B, H, HK, NQ, NK, D, splits):
    assert skl.attn_fwd_plan(B, H, HK, NQ, NK, D, 152)[1] == splits


@pytest.mark.parametrize("NQ,H,HK,B,NK", [(1, 32, 8, 8, 131072), (1, 8, 8, 1, 131072), (4, 32, 8, 1, 4096), (300, 4, 4, 1, 65536)])
def test_splits_come_out_in_whole_waves(NQ, H, HK, B, NK):
    """The waves that the chosen splits take are as full as those of any count near it: a split more, and a wave would start for
    the sake of a few blocks."""
    packed, splits = skl.attn_fwd_plan(B, H, HK, NQ, NK, 128, 152)
    items = B * (HK if packed else H * -(-NQ // 256))
    tiles = -(-NK // 128)

    def cost(s):  # waves of blocks, each as long as its tiles and its set-up
        return -(-items * s // 152) * (-(-tiles // s) + 3)

    assert 1 < splits <= tiles and items * splits <= 4 * 152
    assert cost(splits) <= cost(1)
    assert cost(splits) <= min(cost(s) for s in (splits - 1, splits + 1) if 1 < s <= tiles) + 3
