"""Bounded waits of the dense kernels that run out: the call is reported, ends with
nothing in flight, and the next one is right again."""
import pytest
import torch

import packed_mxfp4_w4a16_b200 as moe
from dense_util import normal
from test_gpu_dense import adapter_inputs, gated_inputs

pytestmark = pytest.mark.gpu

DEFAULT = 1 << 22


@pytest.fixture(autouse=True)
def default_limit():
    yield
    moe.moe_dense_set_spin_limit(DEFAULT)


def check(run):
    want = run()
    torch.cuda.synchronize()
    assert moe.moe_dense_status() == 0
    # no poll at all: every wait gives up; a few polls: some do
    for polls in (0, 1, 3):
        moe.moe_dense_set_spin_limit(polls)
        got = run()
        torch.cuda.synchronize()
        moe.moe_dense_set_spin_limit(DEFAULT)
        status = moe.moe_dense_status()
        assert status in (0, moe.DEVICE_TIMEOUT)
        if polls == 0:
            assert status == moe.DEVICE_TIMEOUT
        if status == 0:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        again = run()
        torch.cuda.synchronize()
        assert moe.moe_dense_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(again, want))


# weights streamed with several ring passes; single CTAs, splits of K; CTA pairs
@pytest.mark.parametrize("T,H,I", [(1, 2048, 7168), (7, 6000, 2056), (20, 4096, 264), (300, 1000, 520),
                                   (2600, 1032, 1544)])
def test_gated(T, H, I):
    x, wg, wu = gated_inputs(T, H, I, seed=T)
    check(lambda: [moe.moe_gated_ffn(x, wg, wu)])


@pytest.mark.parametrize("T,H,I", [(70, 1000, 520), (2600, 1032, 1544)])
def test_backward(T, H, I):
    x, wg, wu = gated_inputs(T, H, I, seed=T)
    dh = normal((T, I), 0.1, T + 5)
    check(lambda: moe.moe_gated_ffn_backward(x, wg, wu, dh))


@pytest.mark.parametrize("T,K,N,rank,n", [(3, 7168, 2048, 16, 5), (33, 136, 72, 24, 3), (64, 7168, 2048, 64, 33),
                                          (129, 2048, 264, 40, 5), (129, 264, 264, 256, 300),
                                          (1030, 264, 1032, 64, 1030), (2561, 264, 2048, 40, 30)])
def test_adapter_proj(T, K, N, rank, n):
    d = adapter_inputs(T, K, N, rank, n, False, seed=T)
    check(lambda: [moe.moe_adapter_proj(**d)])


def test_slow_inner_products_are_no_timeout():
    """A pair's first two tiles name no adapter while the inner products of another
    tile take longer than a bounded wait: nothing waits for them in such a wait."""
    T, K, N, rank, n = 7680, 4104, 1032, 64, 1030
    plan = moe.moe_adapter_proj_plan(T, K, N, n, rank)
    assert plan["products"] == "pairs" and plan["inner"] == "named"
    d = dict(x=normal((T, K), 0.5, 1), w=normal((N, K), 0.02, 2), lora_a=normal((n, rank, K), K ** -0.5, 3),
             lora_b=normal((n, N, rank), 0.05, 4), lora_scale=torch.ones(n, device="cuda"))
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    ids[-128:] = torch.arange(128, dtype=torch.int32, device="cuda") * 8
    want = moe.moe_adapter_proj(**d, adapter_ids=ids)
    torch.cuda.synchronize()
    assert moe.moe_dense_status() == 0
    # about 0.6 ms: the projection's longest tile takes 0.2, the inner products of
    # 128 adapters in one row tile 1.1
    moe.moe_dense_set_spin_limit(400)
    for _ in range(3):
        got = moe.moe_adapter_proj(**d, adapter_ids=ids)
        torch.cuda.synchronize()
        assert moe.moe_dense_status() == 0
        assert torch.equal(got, want)
