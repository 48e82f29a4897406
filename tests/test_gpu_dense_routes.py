"""Projections with adapters on the ways that a call's sizes choose."""
import pytest
import torch

import packed_mxfp4_w4a16_b200 as moe
from test_gpu_dense import adapter_inputs

pytestmark = pytest.mark.gpu


# inner products of every adapter at once, v B^T by plain products
@pytest.mark.parametrize("T,K,N,rank,n", [(64, 7168, 2048, 64, 33), (32, 7168, 2048, 128, 33),
                                          (433, 7912, 272, 8, 3), (426, 312, 296, 128, 7), (257, 264, 392, 136, 4)])
def test_ids_out_of_range_are_reported(T, K, N, rank, n):
    d = adapter_inputs(T, K, N, rank, n, False, seed=T)
    moe.moe_dense_status()
    for at, bad in ((0, n), (T // 2, -2), (T - 1, 2 ** 31 - 1), (T - 1, -2 ** 31)):
        ids = d["adapter_ids"].clone()
        ids[at] = -1
        want = moe.moe_adapter_proj(**dict(d, adapter_ids=ids))
        assert moe.moe_dense_status() == 0
        ids[at] = bad
        assert torch.equal(moe.moe_adapter_proj(**dict(d, adapter_ids=ids)), want)
        assert moe.moe_dense_status() == moe.DEVICE_BAD_ADAPTER_ID, (at, bad)
