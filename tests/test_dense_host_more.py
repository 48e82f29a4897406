"""More host-side checks of the dense feed-forward calls."""
import pytest

import packed_mxfp4_w4a16_b200 as moe


def test_spin_limit_refusal():
    with pytest.raises(moe.MoEError):
        moe.moe_dense_set_spin_limit(-1)
    moe.moe_dense_set_spin_limit(1 << 22)
