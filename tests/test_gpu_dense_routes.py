"""Projections with adapters on the ways that a call's sizes choose."""
import pytest
import torch

import packed_mxfp4_w4a16_b200 as moe
from dense_util import assert_within, gated64
from test_gpu_dense import adapter_inputs, check_adapter, gated_inputs

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


# (T, K, N, adapters, rank), and what their sizes choose: tiles of the projection,
# whether clusters split its K; inner products, whether clusters split theirs;
# whether v B^T comes from plain products
ROUTES = [
    ((3, 7168, 2056, 5, 16), ("streamed", False, "loads", False, True)),
    ((18, 8, 8, 1, 24), ("single", False, "loads", False, False)),
    ((16, 8, 8, 5, 136), ("single", False, "loads", False, True)),
    ((86, 904, 8, 1, 136), ("single", True, "loads", False, False)),
    ((123, 848, 8, 10, 136), ("single", True, "loads", False, True)),
    ((129, 2048, 264, 5, 40), ("single", True, "loads", False, False)),
    ((947, 8, 8, 1, 64), ("single", False, "every", False, False)),
    ((1306, 8, 8, 7, 24), ("single", False, "every", False, True)),
    ((135, 1248, 768, 1, 136), ("single", False, "every", True, False)),
    ((3819, 824, 24, 1, 16), ("single", False, "every", True, True)),
    ((280, 616, 8, 2, 72), ("single", True, "every", False, False)),
    ((635, 552, 8, 11, 64), ("single", True, "every", False, True)),
    ((230, 1064, 8, 1, 72), ("single", True, "every", True, False)),
    ((56, 4376, 24, 36, 200), ("single", True, "every", True, True)),
    ((1696, 8, 256, 1167, 72), ("single", False, "named", False, False)),
    ((3631, 8, 192, 231, 200), ("single", False, "named", False, False)),
    ((129, 264, 264, 300, 256), ("single", False, "named", False, True)),
    ((1176, 8, 8, 931, 72), ("single", False, "named", False, True)),
    ((3792, 640, 72, 550, 24), ("single", False, "named", True, False)),
    ((2330, 544, 8, 112, 72), ("single", False, "named", True, True)),
    ((831, 1656, 8, 99, 64), ("single", True, "named", True, False)),
    ((1742, 1640, 8, 20, 200), ("single", True, "named", True, False)),
    ((1916, 600, 8, 74, 136), ("single", True, "named", True, True)),
    ((374, 8, 8, 18, 16), ("pairs", False, "every", False, False)),
    ((746, 720, 2248, 2, 8), ("pairs", False, "every", True, False)),
    ((1030, 264, 1032, 1030, 64), ("pairs", False, "named", False, False)),
    ((1030, 264, 1032, 200, 136), ("pairs", False, "named", False, False)),
    ((1105, 512, 1256, 106, 200), ("pairs", False, "named", True, False)),
]


@pytest.mark.parametrize("size,route", ROUTES)
def test_every_way_is_right_and_keeps_adapters_apart(size, route):
    T, K, N, n, rank = size
    p = moe.moe_adapter_proj_plan(*size)
    assert (p["products"], p["splits"] > 1, p["inner"], p["inner_splits"] > 1, p["direct"]) == route
    moe.moe_dense_status()
    d = adapter_inputs(T, K, N, rank, n, T % 2 == 1, seed=T)
    ids = d["adapter_ids"]
    ids[T // 2] = broken = n // 2
    clean = check_adapter(d, f"y {size}")
    # non-finite elements of one adapter's B, then of its A
    mine = ids == broken
    touched = torch.zeros(N, dtype=torch.bool, device="cuda")
    touched[[0, N // 2, N - 1]] = True
    b = d["lora_b"]
    b[broken, 0, 0], b[broken, N // 2, rank // 2], b[broken, N - 1, rank - 1] = torch.tensor(
        [float("inf"), float("nan"), -float("inf")], device="cuda").to(torch.bfloat16)
    y = moe.moe_adapter_proj(**d)
    assert torch.equal(y[~mine], clean[~mine])
    assert torch.equal(y[mine][:, ~touched], clean[mine][:, ~touched])
    assert not torch.isfinite(y[mine][:, touched]).any()
    d["lora_a"][broken, rank - 1, K - 1] = float("nan")
    y = moe.moe_adapter_proj(**d)
    assert torch.equal(y[~mine], clean[~mine]) and not torch.isfinite(y[mine]).any()
    assert moe.moe_dense_status() == 0
    # an id behind the pool's last, among others
    want = moe.moe_adapter_proj(**dict(d, adapter_ids=ids.masked_fill(mine, -1)))
    assert moe.moe_dense_status() == 0
    assert torch.equal(moe.moe_adapter_proj(**dict(d, adapter_ids=ids.masked_fill(mine, n))), want)
    assert moe.moe_dense_status() == moe.DEVICE_BAD_ADAPTER_ID
    assert torch.isfinite(want).all()


# K elements of a ring slot: 2048 (several per row), 1024, 512, and tokens that do
# not fit beside any; rows: one tile per CTA or several, so that the ring's passes
# run on from tile to tile
@pytest.mark.parametrize("rows", [8, 264, 5000])
@pytest.mark.parametrize("T,K,streamed", [(1, 2056, True), (1, 7168, True), (4, 6152, True), (8, 5000, True),
                                          (8, 7168, True), (5, 14336, True), (8, 11000, True), (1, 65536, True),
                                          (8, 12000, False), (2, 65536, False)])
def test_few_tokens_of_long_rows(T, K, streamed, rows):
    assert (moe.moe_adapter_proj_plan(T, K, rows, 3, 16)["products"] == "streamed") == streamed
    x, wg, wu = gated_inputs(T, K, rows, seed=K + T)
    assert_within(moe.moe_gated_ffn(x, wg, wu), *gated64(x, wg, wu, "silu"), "h")
    del wg, wu
    d = adapter_inputs(T, K, rows, 16, 3, False, seed=K)
    check_adapter(d, "y")
    check_adapter({k: d[k] for k in ("x", "w")}, "plain")
