"""More host-side checks of the dense feed-forward calls."""
import math
import random

import pytest
import torch

import packed_mxfp4_w4a16_b200 as moe


def test_spin_limit_refusal():
    with pytest.raises(moe.MoEError):
        moe.moe_dense_set_spin_limit(-1)
    moe.moe_dense_set_spin_limit(1 << 22)


def test_plan_refusals_and_the_smallest_calls():
    ctas = (148, 144, 128)
    for bad in (dict(T=0), dict(T=-1), dict(K=12), dict(rank=9), dict(n_adapters=-1), dict(num_sms=-1),
                dict(cluster_ctas=None), dict(num_sms=0)):
        with pytest.raises(moe.MoEError):
            moe.moe_adapter_proj_plan(**{**dict(T=20, K=64, N=32, n_adapters=2, rank=8, num_sms=148,
                                               cluster_ctas=ctas), **bad})
    p = moe.moe_adapter_proj_plan(8, 64, 32, num_sms=148, cluster_ctas=ctas)
    assert p["products"] == "streamed" and p["inner"] == "none" and not p["direct"]
    p = moe.moe_adapter_proj_plan(9, 64, 32, 2, 8, num_sms=148, cluster_ctas=ctas)
    assert p["products"] == "single" and p["inner"] == "loads"
    # few tokens that do not fit in shared memory beside the weights
    assert moe.moe_adapter_proj_plan(8, 40000, 64, num_sms=148, cluster_ctas=ctas)["products"] == "single"


@pytest.mark.parametrize("ctas", [(0, 0, 0), (148, 0, 0), (146, 140, 0), (148, 144, 128)])
def test_only_clusters_that_fit_are_planned(ctas):
    most = max([1] + [2 << i for i in range(3) if ctas[i]])
    rng = random.Random(5)
    pick = lambda lo, hi, step: max(step, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step)
    seen = set()
    for _ in range(3000):
        n, rank = pick(1, 1200, 1), rng.choice([8, 16, 24, 64, 136, 256])
        p = moe.moe_adapter_proj_plan(pick(1, 9000, 1), pick(8, 9000, 8), pick(8, 9000, 8), n, rank, num_sms=148,
                                      cluster_ctas=ctas)
        assert p["splits"] <= most and p["inner_splits"] <= most
        assert p["products"] != "pairs" or most > 1
        seen.add((p["products"], p["inner"], p["direct"]))
    assert {i for _, i, _ in seen} == {"loads", "named", "every"}
    assert ("single", "every", True) in seen and ("single", "named", False) in seen


class NoCalls:
    """In the library's place: a call that gets this far fails the test."""

    def __getattr__(self, name):
        if name == "moe_status_string":
            return moe._lib.load().moe_status_string
        raise AssertionError(f"{name} was called")


BIG = 2 ** 32 + 8  # 8 in 32 bits


def test_sizes_past_32_bits_are_refused(monkeypatch):
    """Integers that do not fit the C calls are refused, not cut to 32 bits."""
    for call in (lambda v: moe.moe_gated_ffn_backward_workspace_bytes(v, 64, 40),
                 lambda v: moe.moe_gated_ffn_backward_workspace_bytes(8, v, 40),
                 lambda v: moe.moe_adapter_proj_workspace_bytes(v, 64, 32, 2, 8),
                 lambda v: moe.moe_adapter_proj_workspace_bytes(8, 64, 32, v, 8),
                 lambda v: moe.moe_adapter_proj_plan(v, 64, 32, num_sms=148, cluster_ctas=(148, 144, 128)),
                 lambda v: moe.moe_dense_set_spin_limit(v)):
        for v in (BIG, -2 ** 32 + 8):
            with pytest.raises(moe.MoEError):
                call(v)
    # tensors of that many rows, without memory behind them
    monkeypatch.setattr(moe, "load", NoCalls)
    t = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device="meta")
    for call in (lambda: moe.moe_gated_ffn(t(BIG, 8), t(8, 8), t(8, 8)),
                 lambda: moe.moe_gated_ffn(t(1, 8), t(BIG, 8), t(BIG, 8)),
                 lambda: moe.moe_gated_ffn_backward(t(BIG, 8), t(8, 8), t(8, 8), t(BIG, 8)),
                 lambda: moe.moe_adapter_proj(t(BIG, 8), t(8, 8)),
                 lambda: moe.moe_adapter_proj(t(1, BIG), t(8, BIG))):
        with pytest.raises(moe.MoEError):
            call()


def test_plan_for_the_smallest_devices():
    """More CTAs than SMs are refused; a single SM has no pairs."""
    for ctas in ((2, 0, 0), (0, 0, 8), (-1, 0, 0)):
        with pytest.raises(moe.MoEError):
            moe.moe_adapter_proj_plan(300, 64, 32, 2, 8, num_sms=1, cluster_ctas=ctas)
    for sms, ctas in ((1, (0, 0, 0)), (1, (1, 1, 1)), (2, (2, 0, 0)), (7, (6, 4, 0))):
        for T in (1, 20, 129, 5000, 2 ** 30):
            for n, rank in ((0, 0), (1, 8), (300, 256), (2 ** 31 - 1, 8)):
                p = moe.moe_adapter_proj_plan(T, 65536, 8, n, rank, num_sms=sms, cluster_ctas=ctas)
                assert sms > 1 or (p["products"] != "pairs" and p["splits"] == 1)
